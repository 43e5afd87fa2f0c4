// Short causal convolution over the channels of a Mamba2 layer: whole packed
// sequences (forward, backward) and one decode step.
//
//   v_t = bias + sum_j w_j x_{t-(W-1)+j},  y_t = silu(v_t)  (or v_t)
//
// Channels are contiguous, so a lane owns eight of them (16 bytes of bf16) and
// walks along the tokens with the window in registers: every x row is read
// once per run of tokens, plus W-1 rows where a run starts.  All of it is
// memory bound (2 W flops per 4 bytes).  5376 channels, W 4, bf16: 16383 tokens
// forward 76 us (0.35 GB, 4.6 TB/s), 16384 backward 124 us (0.53 GB, 4.3 TB/s),
// 512 decode rows 11 us (44 MB, 4.0 TB/s).
#include "rssm_host.hpp"
#include "seq_device.hpp"

namespace rssm {

struct ConvArgs {
  const void* x;
  const float* weight;
  const float* bias;
  const int32_t* cu;
  const void* init;
  const uint8_t* has_init;
  const int32_t* slot_idx;
  void* final_state;
  void* y;
  const void* dy;
  void* dx;
  void* dinit;
  float* part;
  float* dweight;
  float* dbias;
  int32_t* status;
  long x_stride, dy_stride;
  int32_t tokens, seqs, channels, num_slots, silu;
  int32_t run;    // tokens of a wave
  int32_t parts;  // backward: workgroups along the tokens
};

constexpr int kBwdWaves = 4;  // runs of one backward workgroup
constexpr int kBwdChan = 4;   // channels of a lane there
constexpr int kStepRows = 4;  // batch rows of a wave of a large decode step

// The weights of K channels: K W consecutive floats.
template <int W, int K>
struct Taps {
  float w[W][K], b[K];
  __device__ inline void load(const ConvArgs& a, int c0, int n) {
    if (n == K) {
      typedef f32x4 f32x4_any __attribute__((aligned(4)));
      float f[W * K];
      const float* const q = a.weight + (long)c0 * W;
#pragma unroll
      for (int v = 0; v < W * K; v += 4) {
        const f32x4 x = *reinterpret_cast<const f32x4_any*>(q + v);
#pragma unroll
        for (int r = 0; r < 4; ++r) f[v + r] = x[r];
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        b[k] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][k] = f[k * W + j];
      }
      if (a.bias) {
#pragma unroll
        for (int k = 0; k < K; k += 4) {
          const f32x4 x = *reinterpret_cast<const f32x4_any*>(a.bias + c0 + k);
#pragma unroll
          for (int r = 0; r < 4; ++r) b[k + r] = x[r];
        }
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      b[k] = a.bias && k < n ? a.bias[c0 + k] : 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][k] = k < n ? a.weight[(long)(c0 + k) * W + j] : 0.f;
    }
  }
  // v of the window h[0..W-1] (oldest first), lane's k-th channel
  __device__ inline float dot(const float (&h)[W][K], int k) const {
    float v = b[k];
#pragma unroll
    for (int j = 0; j < W; ++j) v = fmaf(w[j][k], h[j][k], v);
    return v;
  }
};

// The slot of sequence i, or -1 (and the status bit) when it is out of range.
__device__ static inline int conv_slot(const ConvArgs& a, int i) {
  const int s = a.slot_idx ? a.slot_idx[i] : i;
  if (s >= 0 && s < a.num_slots) return s;
  if (a.status) atomicOr(a.status, RSSM_ST_BAD_SLOT);
  return -1;
}

// Forward.  Grid: (channel blocks of 64 lanes) x (seqs + runs).  The first
// `seqs` tiles take one sequence's first W-1 tokens and its final state, so
// that every read of an initial state and the write of the final one are the
// same lane's, in that order, and the two may be one pool.  The others take a
// run of tokens and skip the first W-1 of each sequence.
template <typename T, int W>
__global__ void __launch_bounds__(64) conv_fwd_kernel(const ConvArgs a) {
  const int cblocks = (a.channels + 511) / 512;
  // a contiguous range of runs per XCD: the rows two runs share stay in one L2
  const int id = xcd_tile(blockIdx.x, gridDim.x);
  const int tile = id / cblocks, c0 = (id % cblocks) * 512 + threadIdx.x * 8;
  if (c0 >= a.channels) return;
  const int n = a.channels - c0 < 8 ? a.channels - c0 : 8;
  Taps<W, 8> tp;
  tp.load(a, c0, n);
  float h[W][8];
  const auto emit = [&](long t) {
    float o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float v = tp.dot(h, k);
      o[k] = a.silu ? v * sigmoid_f32(v) : v;
    }
    store8<T>(a.y, t * a.channels + c0, n, o);
  };
  const auto shift = [&]() {
#pragma unroll
    for (int j = 0; j + 1 < W; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) h[j][k] = h[j + 1][k];
  };
  if (tile < a.seqs) {
    const SeqSpan sp = seq_span(a.cu, tile, a.seqs, a.tokens);
    if (sp.bad && a.status && c0 == 0) atomicOr(a.status, RSSM_ST_BAD_SEQ);
    const bool pool = a.init || a.final_state;
    const int slot = pool ? conv_slot(a, tile) : -1;
    const bool has = a.init && slot >= 0 && (!a.has_init || a.has_init[tile]);
    float s[W][8];  // the W-1 rows before the sequence
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
#pragma unroll
      for (int k = 0; k < 8; ++k) s[j][k] = 0.f;
      if (has) load8<T>(a.init, ((long)slot * (W - 1) + j) * a.channels + c0, n, s[j]);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[j + 1][k] = s[j][k];
    }
#pragma unroll
    for (int p = 0; p < W - 1; ++p) {
      if (p < sp.len) {
        shift();
        load8<T>(a.x, (long)(sp.start + p) * a.x_stride + c0, n, h[W - 1]);
        emit(sp.start + p);
      }
    }
    if (a.final_state && slot >= 0) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        const int p = sp.len - (W - 1) + j;  // < 0: row p + W-1 before the sequence
        float r[8];
        if (p >= 0) {
          load8<T>(a.x, (long)(sp.start + p) * a.x_stride + c0, n, r);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            r[k] = s[0][k];
#pragma unroll
            for (int q = 1; q < W - 1; ++q) r[k] = p + W - 1 == q ? s[q][k] : r[k];
          }
        }
        store8<T>(a.final_state, ((long)slot * (W - 1) + j) * a.channels + c0, n, r);
      }
    }
    return;
  }
  const int t0 = (tile - a.seqs) * a.run;
  const int t1 = a.tokens - t0 > a.run ? t0 + a.run : a.tokens;
  int i = seq_of_token(a.cu, a.seqs, t0);
#pragma unroll
  for (int j = 1; j < W; ++j) {
    const int t = t0 - W + j;
#pragma unroll
    for (int k = 0; k < 8; ++k) h[j][k] = 0.f;
    if (t >= 0) load8<T>(a.x, (long)t * a.x_stride + c0, n, h[j]);
  }
  int t = t0;
  while (t < t1) {
    SeqSpan sp = seq_span(a.cu, i, a.seqs, a.tokens);
    const bool last = i + 1 >= a.seqs;
    int end = last ? t1 : sp.start + sp.len;
    if (end > t1) end = t1;
    const int from = sp.start + W - 1, to = sp.start + sp.len;
    constexpr int U = 4;  // rows in flight
    for (; t < end; t += U) {
      RawK<T, 8> r[U];
      const auto next = [&](int u) {
        shift();
        r[u].get(h[W - 1]);
      };
      if (t >= from && t + U <= to && t + U <= end) {  // nearly all: no conditions
#pragma unroll
        for (int u = 0; u < U; ++u) r[u].load(a.x, (long)(t + u) * a.x_stride + c0, n);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          next(u);
          emit(t + u);
        }
        continue;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t + u < end) r[u].load(a.x, (long)(t + u) * a.x_stride + c0, n);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u < end) {
          next(u);
          if (t + u >= from && t + u < to) emit(t + u);
        }
      }
    }
    t = end;
    if (last) break;
    ++i;
  }
}

// Backward.  dv_t = dy_t silu'(v_t); dx_t = sum_j w_j dv_{t+(W-1)-j};
// dw_j = sum_t dv_t x_{t-(W-1)+j}; db = sum_t dv_t.  A wave walks its run and
// W-1 tokens past it (their dv again, so that waves need nothing from each
// other); the sums over tokens stay in registers, are joined over the
// workgroup's waves in LDS, in wave order, and go to one row of partial sums
// per workgroup, which a second launch adds in row order: the result does not
// depend on timing.  A lane owns four channels: eight would take 232 registers
// and leave two waves a SIMD.
template <typename T, int W>
__global__ void __launch_bounds__(64 * kBwdWaves) conv_bwd_kernel(const ConvArgs a) {
  constexpr int K = kBwdChan, CB = 64 * K;
  __shared__ float red[kBwdWaves][W + 1][64][K + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cblocks = (a.channels + CB - 1) / CB;
  const int id = xcd_tile(blockIdx.x, gridDim.x);
  const int tile = id / cblocks, cb = (id % cblocks) * CB, c0 = cb + lane * K;
  const int n = a.channels - c0 < K ? (a.channels - c0 < 0 ? 0 : a.channels - c0) : K;
  float dw[W][K] = {}, db[K] = {};
  Taps<W, K> tp;
  tp.load(a, c0, n);
  const long from = ((long)tile * kBwdWaves + wave) * a.run;
  if (from < a.tokens && n > 0) {
    const int t0 = (int)from, t1 = a.tokens - t0 > a.run ? t0 + a.run : a.tokens;
    int t = t0;
    for (int i = seq_of_token(a.cu, a.seqs, t0); t < t1 && i < a.seqs; ++i) {
      const SeqSpan sp = seq_span(a.cu, i, a.seqs, a.tokens);
      const int send = sp.start + sp.len;
      const int b = send < t1 ? send : t1;  // this piece: tokens [t, b) of sequence i
      if (b <= t || t < sp.start) continue;
      float h[W][K], g[W][K];  // windows of x and dv, oldest first
      int slot = -1;
      if (t - sp.start < W - 1 && a.init && (!a.has_init || a.has_init[i])) slot = conv_slot(a, i);
#pragma unroll
      for (int j = 1; j < W; ++j) {
        const int p = t - sp.start - W + j;
        RawK<T, K> r;
        r.zero();
        if (p >= 0)
          r.load(a.x, (long)(sp.start + p) * a.x_stride + c0, n);
        else if (slot >= 0)
          r.load(a.init, ((long)slot * (W - 1) + p + W - 1) * a.channels + c0, n);
        r.get(h[j]);
#pragma unroll
        for (int k = 0; k < K; ++k) g[j][k] = 0.f;
      }
      const int stop = b + W - 1;
      constexpr int U = 4;
      RawK<T, K> rx[U], ro[U];
      // token u of the piece; INNER: well inside it
      const auto token = [&](int q, int u, auto inner) {
        constexpr bool INNER = decltype(inner)::value;
#pragma unroll
        for (int j = 0; j + 1 < W; ++j)
#pragma unroll
          for (int k = 0; k < K; ++k) h[j][k] = h[j + 1][k], g[j][k] = g[j + 1][k];
        float o[K], d[K];
        rx[q].get(h[W - 1]);
        ro[q].get(d);  // 0 past the sequence's end
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (a.silu) {
            const float v = tp.dot(h, k), s = sigmoid_f32(v);
            d[k] *= s * fmaf(v, 1.f - s, 1.f);
          }
          g[W - 1][k] = INNER || u < send ? d[k] : 0.f;
          if (INNER || u < b) {
            db[k] += d[k];
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][k] = fmaf(d[k], h[j][k], dw[j][k]);
          }
          float s = 0.f;
#pragma unroll
          for (int j = 0; j < W; ++j) s = fmaf(tp.w[j][k], g[W - 1 - j][k], s);
          o[k] = s;
        }
        if (INNER || u - (W - 1) >= t) store_k<T, K>(a.dx, (long)(u - (W - 1)) * a.channels + c0, n, o);
      };
      for (int u0 = t; u0 < stop; u0 += U) {
        if (u0 >= t + W - 1 && u0 + U <= b) {
#pragma unroll
          for (int q = 0; q < U; ++q) {
            rx[q].load(a.x, (long)(u0 + q) * a.x_stride + c0, n);
            ro[q].load(a.dy, (long)(u0 + q) * a.dy_stride + c0, n);
          }
#pragma unroll
          for (int q = 0; q < U; ++q) token(q, u0 + q, std::true_type{});
          continue;
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
          rx[q].zero();
          ro[q].zero();
          if (u0 + q < stop && u0 + q < send) {
            rx[q].load(a.x, (long)(u0 + q) * a.x_stride + c0, n);
            ro[q].load(a.dy, (long)(u0 + q) * a.dy_stride + c0, n);
          }
        }
#pragma unroll
        for (int q = 0; q < U; ++q)
          if (u0 + q < stop) token(q, u0 + q, std::false_type{});
      }
      t = b;
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    red[wave][W][lane][k] = db[k];
#pragma unroll
    for (int j = 0; j < W; ++j) red[wave][j][lane][k] = dw[j][k];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < (W + 1) * CB; e += 64 * kBwdWaves) {
    const int j = e / CB, c = e % CB;
    if (cb + c < a.channels) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kBwdWaves; ++w) s += red[w][j][c / K][c % K];
      a.part[((long)tile * (W + 1) + j) * a.channels + cb + c] = s;
    }
  }
}

// dweight [C, W] and dbias [C] from the workgroups' partial sums, rows in
// order within each of four quarters; and (tiles past the columns) the
// gradient of the initial states from each sequence's first W-1 tokens.
template <typename T, int W>
__global__ void __launch_bounds__(256) conv_bwd_join_kernel(const ConvArgs a) {
  const long cols = (long)(W + 1) * a.channels;
  const int cblk = (int)((cols + 63) / 64);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (blockIdx.x == 0) check_table(a.cu, a.seqs, a.tokens, a.status);
  if ((int)blockIdx.x < cblk) {
    __shared__ float red[4][64];
    const long col = (long)blockIdx.x * 64 + lane;
    float s = 0.f;
    if (col < cols) {
      const int per = (a.parts + 3) / 4;
      const int r1 = (wave + 1) * per < a.parts ? (wave + 1) * per : a.parts;
#pragma unroll 8
      for (int r = wave * per; r < r1; ++r) s += a.part[(long)r * cols + col];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && col < cols) {
      s = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
      const int j = (int)(col / a.channels), c = (int)(col % a.channels);
      if (j < W) {
        a.dweight[(long)c * W + j] = s;
      } else if (a.dbias) {
        a.dbias[c] = s;
      }
    }
    return;
  }
  // dinit_k = sum_{j<=k} w_j dv_{k-j}, k = 0 .. W-2 (row k lies W-1-k before
  // the sequence)
  const int lanes = (a.channels + 7) / 8;
  const long id = (long)(blockIdx.x - cblk) * 256 + threadIdx.x;
  const int i = (int)(id / lanes), c0 = (int)(id % lanes) * 8;
  if (i >= a.seqs) return;
  const int n = a.channels - c0 < 8 ? a.channels - c0 : 8;
  const SeqSpan sp = seq_span(a.cu, i, a.seqs, a.tokens);
  const int slot = conv_slot(a, i);
  if (slot < 0) return;
  const bool has = !a.has_init || a.has_init[i];
  Taps<W, 8> tp;
  tp.load(a, c0, n);
  float h[W][8], g[W][8] = {};  // g[p]: dv of token p
  const bool live = has && a.init;
#pragma unroll
  for (int j = 1; j < W; ++j) {
#pragma unroll
    for (int k = 0; k < 8; ++k) h[j][k] = 0.f;
    if (live) load8<T>(a.init, ((long)slot * (W - 1) + j - 1) * a.channels + c0, n, h[j]);
  }
#pragma unroll
  for (int p = 0; p < W - 1; ++p) {
    if (p < sp.len && live) {
      float ro[8];
#pragma unroll
      for (int j = 0; j + 1 < W; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) h[j][k] = h[j + 1][k];
      load8<T>(a.x, (long)(sp.start + p) * a.x_stride + c0, n, h[W - 1]);
      load8<T>(a.dy, (long)(sp.start + p) * a.dy_stride + c0, n, ro);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float d = ro[k];
        if (a.silu) {
          const float v = tp.dot(h, k), s = sigmoid_f32(v);
          d *= s * fmaf(v, 1.f - s, 1.f);
        }
        g[p][k] = d;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    float o[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      o[q] = 0.f;
#pragma unroll
      for (int j = 0; j <= k; ++j) o[q] = fmaf(tp.w[j][q], g[k - j][q], o[q]);
    }
    store8<T>(a.dinit, ((long)slot * (W - 1) + k) * a.channels + c0, n, o);
  }
}

// One decode step: the window is the W-1 state rows and x; the state moves on
// by one row.  A lane reads all it needs of its channels before it writes, so
// the new state may be the old one.  A wave takes R rows of the batch, all of
// whose loads are under way at once, with one read of the weights.
template <typename T, int W, int R>
__global__ void __launch_bounds__(64) conv_step_kernel(const ConvArgs a) {
  const int cblocks = (a.channels + 511) / 512;
  const int row0 = blockIdx.x / cblocks * R, c0 = (blockIdx.x % cblocks) * 512 + threadIdx.x * 8;
  if (c0 >= a.channels) return;
  const int n = a.channels - c0 < 8 ? a.channels - c0 : 8;
  int slot[R];
  RawK<T, 8> r[R][W];
#pragma unroll
  for (int q = 0; q < R; ++q) slot[q] = row0 + q < a.tokens ? conv_slot(a, row0 + q) : -1;
#pragma unroll
  for (int q = 0; q < R; ++q) {
    if (row0 + q < a.tokens) r[q][W - 1].load(a.x, (long)(row0 + q) * a.x_stride + c0, n);
    if (slot[q] >= 0) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        r[q][j].load(a.init, ((long)slot[q] * (W - 1) + j) * a.channels + c0, n);
    }
  }
  Taps<W, 8> tp;
  tp.load(a, c0, n);
#pragma unroll
  for (int q = 0; q < R; ++q) {
    if (row0 + q >= a.tokens) break;
    float o[8], h[W][8];
    if (slot[q] >= 0) {
#pragma unroll
      for (int j = 0; j < W; ++j) r[q][j].get(h[j]);
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        store8<T>(a.final_state, ((long)slot[q] * (W - 1) + j) * a.channels + c0, n, h[j + 1]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = tp.dot(h, k);
        o[k] = a.silu ? v * sigmoid_f32(v) : v;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = __builtin_nanf("");
    }
    store8<T>(a.y, (long)(row0 + q) * a.channels + c0, n, o);
  }
}
template <typename T, int W>
static const void* pick_step(int rows) {
  return rows == 1 ? reinterpret_cast<const void*>(&conv_step_kernel<T, W, 1>)
                   : reinterpret_cast<const void*>(&conv_step_kernel<T, W, kStepRows>);
}

static int conv_check(const rssm_conv_dims* d) {
  if (!d) return RSSM_EINVAL;
  if (d->tokens < 0 || d->seqs < 0 || d->channels < 1 || d->num_slots < 0) return RSSM_EINVAL;
  if (d->activation != RSSM_ACT_NONE && d->activation != RSSM_ACT_SILU) return RSSM_EINVAL;
  if (!valid_dtype(d->io_dtype)) return RSSM_EDTYPE;
  if (d->width < 2 || d->width > 4 || d->channels > (1 << 24)) return RSSM_ESHAPE;
  return RSSM_OK;
}

static bool elt_aligned(const void* p, int32_t dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == RSSM_F32 ? 3u : 1u)) == 0;
}

// Whether any of the rows in[0..rows) (stride apart) shares memory with the dense
// rows out[0..rows), channels of either io_dtype elements: workgroups read up to
// W-1 rows that another one's results would replace.
static bool rows_meet(const void* in, long stride, const void* out, const rssm_conv_dims& d) {
  const long es = d.io_dtype == RSSM_F32 ? 4 : 2, len = d.channels * es;
  return rows_meet(in, stride * es, len, d.tokens, out, d.tokens * len);
}

#define RSSM_CONV_PICK(name, d)                                                        \
  ((d).io_dtype == RSSM_F32                                                            \
       ? ((d).width == 2   ? reinterpret_cast<const void*>(&name<float, 2>)            \
          : (d).width == 3 ? reinterpret_cast<const void*>(&name<float, 3>)            \
                           : reinterpret_cast<const void*>(&name<float, 4>))           \
       : ((d).width == 2   ? reinterpret_cast<const void*>(&name<bf16, 2>)             \
          : (d).width == 3 ? reinterpret_cast<const void*>(&name<bf16, 3>)             \
                           : reinterpret_cast<const void*>(&name<bf16, 4>)))

// Tokens of a wave's run, given the blocks of channels: 32, or less where that
// leaves a SIMD fewer than two waves (a run's first rows are read by two waves,
// which costs a large call more than it gives; 64 is no faster there).  2000 tokens
// of 2000 channels: forward 12.3 us (14.6 with 32), backward 20.7 (25.1).
static int conv_run(const rssm_conv_dims& d, int channels_per_wave) {
  const long cblocks = (d.channels + channels_per_wave - 1) / channels_per_wave;
  int run = 32;
  while (run > 8 && ((long)d.tokens + run - 1) / run * cblocks < 2048) run >>= 1;
  return run;
}
static int bwd_run(const rssm_conv_dims& d) { return conv_run(d, 64 * kBwdChan); }
static long bwd_tiles(const rssm_conv_dims& d) {
  const long per = (long)bwd_run(d) * kBwdWaves;
  return (d.tokens + per - 1) / per;
}

}  // namespace rssm

using namespace rssm;

static ConvArgs conv_args(const rssm_conv_dims& d) {
  ConvArgs a{};
  a.x_stride = d.x_stride ? d.x_stride : d.channels;
  a.dy_stride = d.dy_stride ? d.dy_stride : d.channels;
  a.tokens = d.tokens;
  a.seqs = d.seqs;
  a.channels = d.channels;
  a.num_slots = d.num_slots;
  a.silu = d.activation == RSSM_ACT_SILU;
  return a;
}

extern "C" int causal_conv_forward(const rssm_conv_dims* dims, const void* x, const float* weight,
                                   const float* bias, const int32_t* cu_seqlens,
                                   const void* initial_state, const uint8_t* has_initial,
                                   const int32_t* slot_idx, void* final_state, void* y,
                                   int32_t* status, hipStream_t stream) {
  int rc = conv_check(dims);
  if (rc) return rc;
  const rssm_conv_dims& d = *dims;
  if (d.seqs == 0) return d.tokens == 0 ? RSSM_OK : RSSM_EINVAL;
  const int run = conv_run(d, 512);
  const long grid = (d.seqs + ((long)d.tokens + run - 1) / run) * ((d.channels + 511) / 512);
  if (!grid_fits(grid, 64)) return RSSM_ESHAPE;
  if (!weight || (d.tokens > 0 && (!x || !y))) return RSSM_EINVAL;
  if (!cu_seqlens && d.seqs != 1) return RSSM_EINVAL;
  if (x && (d.x_stride != 0 && d.x_stride < d.channels)) return RSSM_EINVAL;
  if (!elt_aligned(x, d.io_dtype) || !elt_aligned(y, d.io_dtype) ||
      !elt_aligned(initial_state, d.io_dtype) || !elt_aligned(final_state, d.io_dtype))
    return RSSM_EINVAL;
  ConvArgs a = conv_args(d);
  if (rows_meet(x, a.x_stride, y, d)) return RSSM_EINVAL;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.cu = cu_seqlens;
  a.init = initial_state;
  a.has_init = has_initial;
  a.slot_idx = slot_idx;
  a.final_state = final_state;
  a.y = y;
  a.status = status;
  a.run = run;
  return launch_kernel(RSSM_CONV_PICK(conv_fwd_kernel, d), (unsigned)grid, 64, 0, stream, a);
}

extern "C" size_t causal_conv_backward_workspace(const rssm_conv_dims* dims) {
  if (conv_check(dims)) return 0;
  return (size_t)bwd_tiles(*dims) * (dims->width + 1) * dims->channels * sizeof(float);
}

extern "C" int causal_conv_backward(const rssm_conv_dims* dims, const void* dy, const void* x,
                                    const float* weight, const float* bias,
                                    const int32_t* cu_seqlens, const void* initial_state,
                                    const uint8_t* has_initial, const int32_t* slot_idx, void* dx,
                                    float* dweight, float* dbias, void* dinitial_state,
                                    void* workspace, size_t workspace_bytes, int32_t* status,
                                    hipStream_t stream) {
  int rc = conv_check(dims);
  if (rc) return rc;
  const rssm_conv_dims& d = *dims;
  const long parts = bwd_tiles(d), grid = parts * ((d.channels + 64 * kBwdChan - 1) / (64 * kBwdChan));
  const long cols = (long)(d.width + 1) * d.channels;
  const long init = dinitial_state ? ((long)d.seqs * ((d.channels + 7) / 8) + 255) / 256 : 0;
  if (!grid_fits(grid, 64 * kBwdWaves) || !grid_fits((cols + 63) / 64 + init, 256)) return RSSM_ESHAPE;
  if (!weight || !dweight) return RSSM_EINVAL;
  if (d.tokens > 0 && (!x || !dy || !dx || !workspace || d.seqs < 1)) return RSSM_EINVAL;
  if (!cu_seqlens && d.seqs > 1) return RSSM_EINVAL;
  if ((d.x_stride != 0 && d.x_stride < d.channels) ||
      (d.dy_stride != 0 && d.dy_stride < d.channels))
    return RSSM_EINVAL;
  if (!elt_aligned(x, d.io_dtype) || !elt_aligned(dy, d.io_dtype) || !elt_aligned(dx, d.io_dtype) ||
      !elt_aligned(initial_state, d.io_dtype) || !elt_aligned(dinitial_state, d.io_dtype))
    return RSSM_EINVAL;
  if (workspace_bytes < causal_conv_backward_workspace(dims)) return RSSM_EINVAL;
  ConvArgs a = conv_args(d);
  if (rows_meet(x, a.x_stride, dx, d) || rows_meet(dy, a.dy_stride, dx, d)) return RSSM_EINVAL;
  a.x = x;
  a.dy = dy;
  a.weight = weight;
  a.bias = bias;
  a.cu = cu_seqlens;
  a.init = initial_state;
  a.has_init = has_initial;
  a.slot_idx = slot_idx;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.dinit = dinitial_state;
  a.part = static_cast<float*>(workspace);
  a.status = status;
  a.run = bwd_run(d);
  a.parts = (int32_t)parts;
  if (a.parts > 0) {
    rc = launch_kernel(RSSM_CONV_PICK(conv_bwd_kernel, d), (unsigned)grid, 64 * kBwdWaves, 0, stream, a);
    if (rc) return rc;
  }
  return launch_kernel(RSSM_CONV_PICK(conv_bwd_join_kernel, d),
                       (unsigned)((cols + 63) / 64 + init), 256, 0, stream, a);
}

extern "C" int causal_conv_decode(const rssm_conv_dims* dims, const void* x,
                                  const void* conv_state, const float* weight, const float* bias,
                                  const int32_t* slot_idx, void* new_state, void* y,
                                  int32_t* status, hipStream_t stream) {
  int rc = conv_check(dims);
  if (rc) return rc;
  const rssm_conv_dims& d = *dims;
  if (d.tokens == 0) return RSSM_OK;
  // several rows a wave where that still leaves one for every SIMD (512 rows of
  // 5376 channels: 11 us with four, 26 with one and element-wise weight loads)
  const long cblocks = (d.channels + 511) / 512;
  const int rows = d.tokens * cblocks >= 1024 * kStepRows ? kStepRows : 1;
  const long grid = ((long)d.tokens + rows - 1) / rows * cblocks;
  if (!grid_fits(grid, 64)) return RSSM_ESHAPE;
  if (!x || !conv_state || !weight || !new_state || !y) return RSSM_EINVAL;
  if (d.x_stride != 0 && d.x_stride < d.channels) return RSSM_EINVAL;
  if (!elt_aligned(x, d.io_dtype) || !elt_aligned(y, d.io_dtype) ||
      !elt_aligned(conv_state, d.io_dtype) || !elt_aligned(new_state, d.io_dtype))
    return RSSM_EINVAL;
  ConvArgs a = conv_args(d);
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.init = conv_state;
  a.slot_idx = slot_idx;
  a.final_state = new_state;
  a.y = y;
  a.status = status;
  const bool f32 = d.io_dtype == RSSM_F32;
  const void* fn = d.width == 2   ? (f32 ? pick_step<float, 2>(rows) : pick_step<bf16, 2>(rows))
                   : d.width == 3 ? (f32 ? pick_step<float, 3>(rows) : pick_step<bf16, 3>(rows))
                                  : (f32 ? pick_step<float, 4>(rows) : pick_step<bf16, 4>(rows));
  return launch_kernel(fn, (unsigned)grid, 64, 0, stream, a);
}
