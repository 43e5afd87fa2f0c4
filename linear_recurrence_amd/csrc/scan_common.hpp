// Shared pieces of the selective scan's forward and backward kernels.
//
// Tokens of a sequence are taken in chunks of 64.  Within a chunk, with a_t
// the running sum of dt*A (inclusive) and S the state before it,
//   y_t   = e^{a_t} S C_t + sum_{s<=t} e^{a_t-a_s} dt_s (C_t.B_s) x_s + D x_t
//   S'    = e^{a_Q} S + sum_s e^{a_Q-a_s} dt_s x_s B_s^T
// so all the work is small dense products for the matrix cores.
//
// Fragments.  Both operands of a 16x16x32 product give lane l the eight
// k-values of its row (A) or column (B) l%16; which k they are is free as long
// as both agree.  Order C: k = 8g + e (g = l/16), contiguous.  Order D:
// k = 4g + e for e < 4 and 16 + 4g + e - 4 above: what a lane holds of a pair
// of 16x16 results (rows 4g + r), so a result becomes an operand without
// moving between lanes.
#pragma once

#include "rssm_host.hpp"
#include "seq_device.hpp"

namespace rssm {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

template <typename T> struct Mat;

template <> struct Mat<bf16> {
  typedef uint16_t E;
  typedef u32x4 Frag;
  static constexpr int kPad = 8;    // elements between LDS rows: rows start 4 banks apart
  static constexpr int kTerms = 3;  // bf16 terms that hold an fp32 value (3 x 8 bits)
  __device__ static inline Frag rows_c(const E* p) { return *reinterpret_cast<const u32x4*>(p); }
  __device__ static inline Frag rows_d(const E* p) {
    const u32x2 a = *reinterpret_cast<const u32x2*>(p);
    const u32x2 b = *reinterpret_cast<const u32x2*>(p + 16);
    return Frag{a[0], a[1], b[0], b[1]};
  }
  // p: row 4g + (l%16)/4 of the K block, the lane's granule of 4 columns; the
  // transposing read hands lane l the 4 rows of column l%16
  __device__ static inline Frag cols(const E* p, int ld) {
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * ld));
    const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
    return Frag{x[0], x[1], y[0], y[1]};
  }
  __device__ static inline f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
    return mfma16x16x32_bf16(a, b, c);
  }
  // one conversion a pair (v_cvt_pk_bf16_f32, to nearest even)
  __device__ static inline Frag pack(const float* f) {
    Frag v;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = bf16_pk(f[2 * k], f[2 * k + 1]);
    return v;
  }
  __device__ static inline void unpack(const Frag& a, float* f) { Elt<bf16>::unpack(a, f); }
  // four neighbours
  typedef u32x2 Four;
  __device__ static inline Four pack4(const float* f) { return Four{bf16_pk(f[0], f[1]), bf16_pk(f[2], f[3])}; }
  __device__ static inline void unpack4(Four v, float* f) {
    f[0] = __uint_as_float(v[0] << 16);
    f[1] = __uint_as_float(v[0] & 0xffff0000u);
    f[2] = __uint_as_float(v[1] << 16);
    f[3] = __uint_as_float(v[1] & 0xffff0000u);
  }
};

template <> struct Mat<float> {
  typedef float E;
  struct Frag {
    float v[8];
  };
  static constexpr int kPad = 4;
  static constexpr int kTerms = 1;
  __device__ static inline Frag rows_c(const E* p) {
    Frag f;
    Elt<float>::unpack(*reinterpret_cast<const u32x4*>(p), f.v);
    Elt<float>::unpack(*reinterpret_cast<const u32x4*>(p + 4), f.v + 4);
    return f;
  }
  __device__ static inline Frag rows_d(const E* p) {
    Frag f;
    Elt<float>::unpack(*reinterpret_cast<const u32x4*>(p), f.v);
    Elt<float>::unpack(*reinterpret_cast<const u32x4*>(p + 16), f.v + 4);
    return f;
  }
  // p: row 4g of the K block, the lane's column
  __device__ static inline Frag cols(const E* p, int ld) {
    Frag f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = p[(e < 4 ? e : 12 + e) * ld];
    return f;
  }
  // fp32 inputs keep fp32 products: eight 16x16x4 steps, step e taking the
  // lanes' e-th values
  __device__ static inline f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
    return c;
  }
  __device__ static inline Frag pack(const float* f) {
    Frag r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = f[e];
    return r;
  }
  __device__ static inline void unpack(const Frag& a, float* f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = a.v[e];
  }
  typedef f32x4 Four;
  __device__ static inline Four pack4(const float* f) { return Four{f[0], f[1], f[2], f[3]}; }
  __device__ static inline void unpack4(Four v, float* f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = v[e];
  }
};

// A lane's address of a column fragment.
template <typename T, bool PAIRED>
__device__ static inline const typename Mat<T>::E* cols_at(const typename Mat<T>::E* tile, int ld,
                                                           int k0, int c0, int lane) {
  return tile + cols_offset<sizeof(typename Mat<T>::E), PAIRED>(ld, k0, c0, lane);
}

// An fp32 operand as kTerms fragments whose sum it is: each product with an
// exact operand is then an fp32 one.
template <typename T, int TERMS>
struct Split {
  typename Mat<T>::Frag t[TERMS];
  __device__ inline void set(const float* f) {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = f[e];
#pragma unroll
    for (int k = 0; k < TERMS; ++k) {
      t[k] = Mat<T>::pack(r);
      if (k + 1 < TERMS) {
        float q[8];
        Mat<T>::unpack(t[k], q);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] -= q[e];
      }
    }
  }
  // this * other (this one the A operand), smallest terms first
  __device__ inline f32x4 a_times(const typename Mat<T>::Frag& o, f32x4 c) const {
#pragma unroll
    for (int k = TERMS - 1; k >= 0; --k) c = Mat<T>::mma(t[k], o, c);
    return c;
  }
  // other * this (this one the B operand)
  __device__ inline f32x4 b_times(const typename Mat<T>::Frag& o, f32x4 c) const {
#pragma unroll
    for (int k = TERMS - 1; k >= 0; --k) c = Mat<T>::mma(o, t[k], c);
    return c;
  }
};

// One row of 16-byte loads from a strided matrix into an LDS tile of kQ rows,
// zero past `rows` (and past `cols` up to the tile's width).
template <typename T, int COLS, int TILE, int THREADS>
__device__ static inline void stage_tile(typename Mat<T>::E* tile, int ld, const void* src,
                                         long stride, int rows, int tid) {
  typedef typename Mat<T>::E E;
  constexpr int V = 16 / sizeof(E), PER = TILE / V;
  constexpr bool kWhole = kQ * PER % THREADS == 0;
#pragma unroll
  for (int q = 0; q < (kQ * PER + THREADS - 1) / THREADS; ++q) {
    const int e = q * THREADS + tid, r = e / PER, c = (e % PER) * V;
    if (!kWhole && e >= kQ * PER) break;
    u32x4 v = {0, 0, 0, 0};
    if (r < rows && (COLS == TILE || c < COLS))
      v = *reinterpret_cast<const u32x4*>(static_cast<const E*>(src) + r * stride + c);
    *reinterpret_cast<u32x4*>(tile + r * ld + c) = v;
  }
}

// The value is unknown from here on: what is worked out from it (addresses,
// conversions) is worked out again in each round of a loop, instead of being
// kept in registers across all of them.
__device__ static inline void forget(int& v) { asm volatile("" : "+v"(v)); }
__device__ static inline void forget(u32x2& v) { asm volatile("" : "+v"(v)); }
__device__ static inline void forget(f32x4& v) { asm volatile("" : "+v"(v)); }

// Nothing is scheduled across this point: fully unrolled, the compiler would
// start every tile's products at once and spill what they leave.
__device__ static inline void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// A wave's own writes to LDS, before its other lanes read them (and its reads,
// before they are written over).
__device__ static inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Inclusive sum over the wave's lanes (0 to 63) in double: decays are
// differences of these sums, and a large step must not cost the small ones
// their digits.
__device__ static inline double wave_cumsum(double v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double t = __shfl_up(v, o, 64);
    if (lane >= o) v += t;
  }
  return v;
}

__device__ static inline float exp2_f32(float v) { return __builtin_amdgcn_exp2f(v); }

// log2 of the decay between two tokens, from their sums as (high, low) pairs.
__device__ static inline float gap2(float2 t, float2 s) { return (t.x - s.x) + (t.y - s.y); }

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
  float* seg_state;  // [slots][V][32][N]
  float* seg_decay;  // [slots][V], log2
  f32x4* dec;        // [chunk slots][H][64]: sum of dt A (log2; high, low), dt, dt before softplus
  void* chunk_state; // [chunk slots][V][32 N], fp32: the state before the chunk
  int32_t* status;
  long x_stride, dt_stride, B_stride, C_stride, z_stride;
  int32_t tokens, seqs, nheads, headdim, dstate, ngroups, num_slots, state_bf16, dt_softplus;
  int32_t seg, vheads, vpg;
  int32_t hb, upb, upg;  // blocks of units in a group, units a block, units a group
};

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

static inline int scan_check(const rssm_scan_dims* d) {
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

// The sizes and strides of the arguments (a stride of 0 is a dense operand).
static inline void fill_dims(ScanArgs& a, const rssm_scan_dims& d) {
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
}

// dt and the running sum of dt*A (log2) of a chunk's tokens, one per lane.
struct ChunkDt {
  float raw, dt;
  double cum, all;
};
template <typename T>
__device__ static inline ChunkDt chunk_dt(const ScanArgs& a, int h, float bias, double A2, long t0,
                                          int rows, int lane) {
  ChunkDt c;
  c.raw = c.dt = 0.f;
  if (lane < rows) {
    c.raw = Elt<T>::load1(a.dt, (t0 + lane) * a.dt_stride + h) + bias;
    c.dt = a.dt_softplus ? softplus_exact(c.raw) : c.raw;
  }
  c.cum = wave_cumsum((double)c.dt * A2, lane);
  c.all = __shfl(c.cum, 63, 64);
  return c;
}

// dt and the running sums of dt*A of one chunk and head, a wave each.
template <typename T>
static __global__ void __launch_bounds__(256) scan_decay_kernel(const ScanArgs a) {
  const int lane = threadIdx.x & 63, hq = (a.nheads + 3) / 4;
  const long slot = blockIdx.x / hq;
  const int h = (int)(blockIdx.x % hq) * 4 + (threadIdx.x >> 6);
  const Segment sg = find_segment(a.cu, a.seqs, a.tokens, kQ, (int)slot);
  if (sg.len == 0 || h >= a.nheads) return;
  const double A2 = (double)a.A[h] * 1.4426950408889634074;
  const ChunkDt q = chunk_dt<T>(a, h, a.dt_bias ? a.dt_bias[h] : 0.f, A2, sg.tok, sg.len, lane);
  const float hi = (float)q.cum;
  a.dec[(slot * a.nheads + h) * kQ + lane] = f32x4{hi, (float)(q.cum - (double)hi), q.dt, q.raw};
}
template <typename T>
static inline int launch_decay(const ScanArgs& a, long cslots, hipStream_t stream) {
  return launch_kernel(reinterpret_cast<const void*>(&scan_decay_kernel<T>),
                       (unsigned)(cslots * ((a.nheads + 3) / 4)), 256, 0, stream, a);
}

__device__ static inline float gap2(f32x4 t, f32x4 s) { return (t[0] - s[0]) + (t[1] - s[1]); }
__device__ static inline f32x4 lane_of(f32x4 v, int l) {
  f32x4 o = v;
  o[0] = __shfl(v[0], l, 64);
  o[1] = __shfl(v[1], l, 64);
  return o;
}

// acc[nt][pt] += (w * rows of X)^T (rows of Y): X the wave's [64][32] tile, Y
// the shared [64][N] one, w one weight per token; ROWS: X's columns are the
// result's rows, otherwise its columns.
template <typename T, int NT, int LX, int LN, bool ROWS>
__device__ static inline void rank_update(f32x4 (&acc)[NT][2], const typename Mat<T>::E* X,
                                          const typename Mat<T>::E* Y, const float* w, int rows,
                                          int lane) {
  typedef Mat<T> M;
  const int g = lane >> 4;
#pragma unroll 1
  for (int kb = 0; kb < kQ / 32; ++kb) {
    if (32 * kb >= rows) break;
    Split<T, M::kTerms> xs[2];
    const float* w0 = w + 32 * kb + 4 * g;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float f[8];
      M::unpack(M::cols(cols_at<T, true>(X, LX, 32 * kb, pair_base(p), lane), LX), f);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        f[r] *= w0[r];
        f[4 + r] *= w0[16 + r];
      }
      xs[p].set(f);
    }
    // two column tiles at a time, the terms outside: four products in a row that
    // do not wait for each other
    constexpr int U = NT < 2 ? 1 : 2;
#pragma unroll
    for (int n = 0; n < NT; n += U) {
      typename M::Frag y[U];
#pragma unroll
      for (int q = 0; q < U; ++q)
        y[q] = M::cols(cols_at<T, false>(Y, LN, 32 * kb, 16 * (n + q), lane), LN);
#pragma unroll
      for (int k = M::kTerms - 1; k >= 0; --k)
#pragma unroll
        for (int q = 0; q < U; ++q)
#pragma unroll
          for (int p = 0; p < 2; ++p)
            acc[n + q][p] = ROWS ? M::mma(xs[p].t[k], y[q], acc[n + q][p])
                                 : M::mma(y[q], xs[p].t[k], acc[n + q][p]);
    }
  }
}

}  // namespace rssm
