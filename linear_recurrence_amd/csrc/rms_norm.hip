// Root-mean-square norm around a Mamba2 layer's blocks: the residual's
// addition, a silu gate, norm groups and an 8-bit output with scales; and its
// backward pass.
//
//   h = x + residual (stored in the residual's type, and read as stored)
//   u = h * silu(z);  y = u * rsqrt(mean_group(u^2) + eps) * weight
//
// Memory bound.  A workgroup owns a row and holds all of it in registers (up
// to 32 elements a lane), so each input is read once.  The row is cut into
// vectors of eight elements that never cross a group's border (a group's last
// vector may be shorter), so any length and any start works with the same
// 16-byte loads.  16383 rows of 2560 with an fp32 residual and e4m3 output 88 us
// (0.46 GB, 5.2 TB/s); 8192 gated rows of 8192 backward 164 us (0.67 GB, 4.1 TB/s).
#include "rssm_host.hpp"
#include "seq_device.hpp"

namespace rssm {

struct NormArgs {
  const void* x;
  const void* z;
  const void* residual;
  const float* weight;
  void* res_out;
  void* out;
  float* scale;
  const void* dy;
  void* dx;
  void* dz;
  float* part;
  float* dweight;
  long x_stride, z_stride, dy_stride;
  float eps, inv_group;
  int32_t rows, dim, group, ngroups, gvec, nvec, res_f32, fp8, scale_block, parts;
};

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;

template <int T>
__device__ static inline float block_sum(float v, float* lds) {
  v = group_sum<64>(v);
  if constexpr (T == 64) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < T / 64; ++w) s += lds[w];
  return s;
}

// The larger value, or NaN if either is one (a scale must not hide a NaN).
__device__ static inline float max_nan(float a, float b) { return b > a || b != b ? b : a; }

template <int W>
__device__ static inline float group_max(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) {
    const float t = __shfl_xor(v, o, 64);
    v = v != v ? v : max_nan(v, t);
  }
  return v;
}

// Sums of each group's vectors from the lanes' per-vector values: through LDS
// when there are several groups (one wave adds one group, lanes in a fixed
// order), a workgroup sum when there is one.  got(v) is then vector v's
// group's sum.
template <int T, int V>
__device__ static inline void group_sums(const NormArgs& a, const float (&s)[V], const int (&g)[V],
                                         float* lds, float (&got)[V]) {
  if (a.ngroups == 1) {
    float t = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) t += s[v];
    t = block_sum<T>(t, lds);
#pragma unroll
    for (int v = 0; v < V; ++v) got[v] = t;
    return;
  }
  float* sums = lds + a.nvec;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int q = v * T + threadIdx.x;
    if (q < a.nvec) lds[q] = s[v];
  }
  __syncthreads();
  const int lane = threadIdx.x & 63;
  for (int k = threadIdx.x >> 6; k < a.ngroups; k += T / 64) {
    float t = 0.f;
    for (int j = lane; j < a.gvec; j += 64) t += lds[k * a.gvec + j];
    t = group_sum<64>(t);
    if (lane == 0) sums[k] = t;
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) got[v] = g[v] < a.ngroups ? sums[g[v]] : 0.f;
}

// The vectors of this lane: group, first element, elements (0: none).
template <int T, int V>
struct Lay {
  int g[V], i[V], n[V];
  __device__ inline void set(const NormArgs& a) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int q = v * T + threadIdx.x;
      g[v] = a.ngroups == 1 ? 0 : q / a.gvec;
      const int j = q - g[v] * a.gvec, left = a.group - 8 * j;
      i[v] = g[v] * a.group + 8 * j;
      n[v] = q < a.nvec ? (left < 8 ? left : 8) : 0;
    }
  }
};

// Four fp32 to four e4m3 bytes, round to nearest even (|f| <= 448).
__device__ static inline uint32_t fp8x4(const float* f) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], r, true);
}

template <typename E, int T, int V>
__global__ void __launch_bounds__(T) norm_fwd_kernel(const NormArgs a) {
  extern __shared__ float lds[];
  const long row = blockIdx.x;
  Lay<T, V> l;
  l.set(a);
  float u[V][8], s[V], tot[V];
#pragma unroll
  for (int v = 0; v < V; ++v) load8<E>(a.x, row * a.x_stride + l.i[v], l.n[v], u[v]);
  if (a.residual) {
    float r[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const long e = row * a.dim + l.i[v];
      if (a.res_f32) load8<float>(a.residual, e, l.n[v], r[v]);
      else load8<E>(a.residual, e, l.n[v], r[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const long e = row * a.dim + l.i[v];
#pragma unroll
      for (int k = 0; k < 8; ++k) u[v][k] += r[v][k];
      if (a.res_f32) {
        store8<float>(a.res_out, e, l.n[v], u[v]);
      } else {
        store8<E>(a.res_out, e, l.n[v], u[v]);
        // the norm reads what the next block will read: the stored value
        if constexpr (sizeof(E) == 2) Elt<bf16>::unpack(Elt<bf16>::pack(u[v]), u[v]);
      }
    }
  }
  if (a.z) {
    float z[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) load8<E>(a.z, row * a.z_stride + l.i[v], l.n[v], z[v]);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int k = 0; k < 8; ++k) u[v][k] *= z[v][k] * sigmoid_f32(z[v][k]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s[v] = fmaf(u[v][k], u[v][k], s[v]);
  }
  group_sums<T, V>(a, s, l.g, lds, tot);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float r = __builtin_amdgcn_rsqf(tot[v] * a.inv_group + a.eps);
    float w[8];
    load8<float>(a.weight, l.i[v], l.n[v], w);
#pragma unroll
    for (int k = 0; k < 8; ++k) u[v][k] = u[v][k] * r * w[k];
  }
  if (!a.fp8) {
#pragma unroll
    for (int v = 0; v < V; ++v) store8<E>(a.out, row * a.dim + l.i[v], l.n[v], u[v]);
    return;
  }
  // scale = max|y| / 448 over the row or over 128 elements (16 lanes: there
  // the group is a multiple of 128, so vectors of a block are consecutive)
  float top[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    top[v] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top[v] = top[v] != top[v] || k >= l.n[v] ? top[v] : max_nan(top[v], fabsf(u[v][k]));
  }
  if (a.scale_block) {
#pragma unroll
    for (int v = 0; v < V; ++v) top[v] = group_max<16>(top[v]);
  } else {
    float t = top[0];
#pragma unroll
    for (int v = 1; v < V; ++v) t = t != t ? t : max_nan(t, top[v]);
    t = group_max<64>(t);
    if constexpr (T > 64) {
      __syncthreads();
      if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = t;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < T / 64; ++w) t = t != t ? t : max_nan(t, lds[w]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) top[v] = t;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    // a scale below the smallest normal number would have no reciprocal
    const float sc = top[v] > 0.f ? fmaxf(top[v] / kE4m3Max, kMinScale) : 1.f;
    const float inv = 1.f / sc;
    if (a.scale_block) {
      if (l.n[v] && (l.i[v] & 127) == 0) a.scale[row * (a.dim / 128) + l.i[v] / 128] = sc;
    } else if (v == 0 && threadIdx.x == 0) {
      a.scale[row] = sc;
    }
    float q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float t = u[v][k] * inv;  // clamped so that a NaN stays one
      q[k] = t > kE4m3Max ? kE4m3Max : (t < -kE4m3Max ? -kE4m3Max : t);
    }
    const u32x2 b = {fp8x4(q), fp8x4(q + 4)};
    uint8_t* o = static_cast<uint8_t*>(a.out) + row * a.dim + l.i[v];
    if (l.n[v] == 8) {
      *reinterpret_cast<u32x2_any*>(o) = b;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < l.n[v]) o[k] = (uint8_t)(b[k >> 2] >> (8 * (k & 3)));
    }
  }
}

// The same for two values a vector at once; a group's sums replace its first
// vector's values.
template <int T, int V>
__device__ static inline void group_sums2(const NormArgs& a, float (&s)[V], float (&d)[V],
                                          const int (&g)[V], float2* lds) {
  const int lane = threadIdx.x & 63;
  if (a.ngroups == 1) {
    float2 t = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) t.x += s[v], t.y += d[v];
    t.x = group_sum<64>(t.x);
    t.y = group_sum<64>(t.y);
    if constexpr (T > 64) {
      __syncthreads();
      if (lane == 0) lds[threadIdx.x >> 6] = t;
      __syncthreads();
      t = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < T / 64; ++w) t.x += lds[w].x, t.y += lds[w].y;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = t.x, d[v] = t.y;
    return;
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int q = v * T + threadIdx.x;
    if (q < a.nvec) lds[q] = make_float2(s[v], d[v]);
  }
  __syncthreads();
  for (int k = threadIdx.x >> 6; k < a.ngroups; k += T / 64) {
    float2 t = make_float2(0.f, 0.f);
    for (int j = lane; j < a.gvec; j += 64) {
      const float2 o = lds[k * a.gvec + j];
      t.x += o.x;
      t.y += o.y;
    }
    t.x = group_sum<64>(t.x);
    t.y = group_sum<64>(t.y);
    if (lane == 0) lds[k * a.gvec] = t;
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float2 t = g[v] < a.ngroups ? lds[g[v] * a.gvec] : make_float2(0.f, 0.f);
    s[v] = t.x;
    d[v] = t.y;
  }
}

// With r = rsqrt(mean(u^2) + eps) and t = dy * weight:
//   du = r (t - u r^2 mean(t u)),  dweight = sum_rows dy u r,
//   dh = du silu(z),  dz = du h silu'(z).
// A workgroup takes every gridDim-th row and keeps its share of dweight in
// registers; one row of partial sums per workgroup, added in order by a
// second launch.  The inputs stay as they are stored (half the registers of
// fp32), and the next row's are on their way while one is worked on.
template <typename E, int T, int V>
__global__ void __launch_bounds__(T) norm_bwd_kernel(const NormArgs a) {
  extern __shared__ float2 lds2[];
  constexpr bool kAhead = V <= 2;
  Lay<T, V> l;
  l.set(a);
  float dw[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[v][k] = 0.f;
  struct Row {
    RawK<E, 8> x[V], o[V], z[V];
    __device__ inline void load(const NormArgs& a, const Lay<T, V>& l, long row) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        x[v].load(a.x, row * a.x_stride + l.i[v], l.n[v]);
        o[v].load(a.dy, row * a.dy_stride + l.i[v], l.n[v]);
        if (a.z) z[v].load(a.z, row * a.z_stride + l.i[v], l.n[v]);
      }
    }
  };
  Row now, next;
  if (kAhead && (long)blockIdx.x < a.rows) next.load(a, l, blockIdx.x);
  for (long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    if constexpr (kAhead) {
      now = next;
      if (row + gridDim.x < a.rows) next.load(a, l, row + gridDim.x);
    } else {
      now.load(a, l, row);
    }
    float s[V], dot[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = dot[v] = 0.f;
      float w[8], x[8], o[8], z[8];
      load8<float>(a.weight, l.i[v], l.n[v], w);
      now.x[v].get(x);
      now.o[v].get(o);
      if (a.z) now.z[v].get(z);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float u = a.z ? x[k] * (z[k] * sigmoid_f32(z[k])) : x[k];
        s[v] = fmaf(u, u, s[v]);
        dot[v] = fmaf(u, o[k] * w[k], dot[v]);
      }
    }
    group_sums2<T, V>(a, s, dot, l.g, lds2);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float r = __builtin_amdgcn_rsqf(s[v] * a.inv_group + a.eps);
      const float c = r * r * (dot[v] * a.inv_group);
      float w[8], x[8], o[8], z[8];
      load8<float>(a.weight, l.i[v], l.n[v], w);
      now.x[v].get(x);
      now.o[v].get(o);
      if (a.z) now.z[v].get(z);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float gate = 1.f, dgate = 0.f;
        if (a.z) {
          const float sg = sigmoid_f32(z[k]);
          gate = z[k] * sg;
          dgate = sg * fmaf(z[k], 1.f - sg, 1.f);
        }
        const float u = x[k] * gate;
        const float du = r * (o[k] * w[k] - u * c);
        dw[v][k] = fmaf(o[k], u * r, dw[v][k]);
        z[k] = du * x[k] * dgate;
        x[k] = du * gate;
      }
      store8<E>(a.dx, row * a.dim + l.i[v], l.n[v], x);
      if (a.z) store8<E>(a.dz, row * a.dim + l.i[v], l.n[v], z);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    store8<float>(a.part, (long)blockIdx.x * a.dim + l.i[v], l.n[v], dw[v]);
}

__global__ void __launch_bounds__(256) norm_bwd_join_kernel(const NormArgs a) {
  __shared__ float red[16][17];
  const int c = threadIdx.x & 15, k = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + c;
  float s = 0.f;
  if (col < a.dim) {
    const int per = (a.parts + 15) / 16;
    const int r1 = (k + 1) * per < a.parts ? (k + 1) * per : a.parts;
#pragma unroll 8
    for (int r = k * per; r < r1; ++r) s += a.part[(long)r * a.dim + col];
  }
  red[k][c] = s;
  __syncthreads();
  if (k == 0 && col < a.dim) {
    s = 0.f;
#pragma unroll
    for (int q = 0; q < 16; ++q) s += red[q][c];
    a.dweight[col] = s;
  }
}

// Threads of a row's workgroup and vectors a lane: rows up to 1024 elements
// take one wave (no barrier), up to 4096 four waves, up to 8192 four (forward)
// or eight (backward, which holds two rows of three tensors), up to 32768
// sixteen.
struct NormShape {
  int threads, vecs;
};
static NormShape norm_shape(int nvec, bool backward, int rows = 1 << 30) {
  // at most one row a compute unit: all of it at once (64 rows of 5120: 6.5 us
  // instead of 8.8)
  if (!backward && rows <= 256 && nvec > 256 && nvec <= 1024) return {1024, 1};
  if (nvec <= 64) return {64, 1};
  if (nvec <= 128) return {64, 2};
  if (nvec <= 256) return {256, 1};
  if (nvec <= 512) return {256, 2};
  if (nvec <= 1024) return backward ? NormShape{512, 2} : NormShape{256, 4};
  if (nvec <= 2048) return {1024, 2};
  return {1024, 4};
}

template <int T, int V>
static bool norm_is(const NormShape& sh) {
  return sh.threads == T && sh.vecs == V;
}
#define RSSM_NORM_CASE(name, E, ...)                                        \
  if (norm_is<__VA_ARGS__>(sh)) return reinterpret_cast<const void*>(&name<E, __VA_ARGS__>)
#define RSSM_NORM_PICK(name, ...)                                               \
  template <typename E>                                                      \
  static const void* pick_##name(const NormShape& sh) {                      \
    RSSM_NORM_CASE(name, E, 64, 1);                                          \
    RSSM_NORM_CASE(name, E, 64, 2);                                          \
    RSSM_NORM_CASE(name, E, 256, 1);                                         \
    RSSM_NORM_CASE(name, E, 256, 2);                                         \
    RSSM_NORM_CASE(name, E, __VA_ARGS__);                                    \
    RSSM_NORM_CASE(name, E, 1024, 2);                                        \
    return reinterpret_cast<const void*>(&name<E, 1024, 4>);                 \
  }
RSSM_NORM_PICK(norm_fwd_kernel, 256, 4)
RSSM_NORM_PICK(norm_bwd_kernel, 512, 2)

static int norm_check(const rssm_norm_dims* d, NormArgs* a) {
  if (!d) return RSSM_EINVAL;
  if (d->rows < 0 || d->dim < 1 || d->group_size < 1 || d->dim % d->group_size) return RSSM_EINVAL;
  if (!(d->eps >= 0.f)) return RSSM_EINVAL;
  if (!valid_dtype(d->io_dtype) || !valid_dtype(d->residual_dtype)) return RSSM_EDTYPE;
  if (d->residual_dtype != RSSM_F32 && d->residual_dtype != d->io_dtype) return RSSM_EDTYPE;
  if (d->out_dtype != RSSM_F8E4M3 && d->out_dtype != d->io_dtype) return RSSM_EDTYPE;
  if ((d->x_stride && d->x_stride < d->dim) || (d->z_stride && d->z_stride < d->dim) ||
      (d->dy_stride && d->dy_stride < d->dim))
    return RSSM_EINVAL;
  const int ng = d->dim / d->group_size;
  const long nvec = (long)ng * ((d->group_size + 7L) / 8);
  if (nvec > 4096) return RSSM_ESHAPE;  // 16 waves with 32 elements a lane
  if (d->out_dtype == RSSM_F8E4M3) {
    if (d->scale_block != 0 && d->scale_block != 128) return RSSM_ESHAPE;
    if (d->scale_block && d->group_size % 128) return RSSM_ESHAPE;
  } else if (d->scale_block) {
    return RSSM_EINVAL;
  }
  a->rows = d->rows;
  a->dim = d->dim;
  a->group = d->group_size;
  a->ngroups = ng;
  a->gvec = (d->group_size + 7) / 8;
  a->nvec = (int32_t)nvec;
  a->eps = d->eps;
  a->inv_group = 1.f / (float)d->group_size;
  a->x_stride = d->x_stride ? d->x_stride : d->dim;
  a->z_stride = d->z_stride ? d->z_stride : d->dim;
  a->dy_stride = d->dy_stride ? d->dy_stride : d->dim;
  a->res_f32 = d->residual_dtype == RSSM_F32;
  a->fp8 = d->out_dtype == RSSM_F8E4M3;
  a->scale_block = d->scale_block;
  return RSSM_OK;
}

// Reductions: one float a vector and one a group when there are several
// groups, one a wave otherwise.
static size_t norm_lds(const NormArgs& a) {
  return a.ngroups > 1 ? sizeof(float) * ((size_t)a.nvec + a.ngroups + 16) : 16 * sizeof(float);
}

static bool elt_aligned(const void* p, bool f32) {
  return (reinterpret_cast<uintptr_t>(p) & (f32 ? 3u : 1u)) == 0;
}

// Workgroups of the backward pass: sixteen waves a compute unit (what their
// registers leave room for), and no more than there are rows.
static int bwd_parts(const NormArgs& a) {
  const int most = 256 * 1024 / norm_shape(a.nvec, true).threads;
  const int cap = most < 2048 ? most : 2048;
  return a.rows < cap ? a.rows : cap;
}
static size_t norm_bwd_lds(const NormArgs& a) {
  return sizeof(float2) * (a.ngroups > 1 ? (size_t)a.nvec : 16);
}

}  // namespace rssm

using namespace rssm;

extern "C" int rms_norm_forward(const rssm_norm_dims* dims, const void* x, const float* weight,
                                const void* z, const void* residual, void* residual_out, void* out,
                                float* scale, hipStream_t stream) {
  NormArgs a{};
  int rc = norm_check(dims, &a);
  if (rc) return rc;
  if (a.rows == 0) return RSSM_OK;
  if (!x || !weight || !out || (residual && !residual_out) || (a.fp8 && !scale))
    return RSSM_EINVAL;
  const bool f32 = dims->io_dtype == RSSM_F32;
  if (!elt_aligned(x, f32) || !elt_aligned(z, f32) || (!a.fp8 && !elt_aligned(out, f32)) ||
      !elt_aligned(residual, a.res_f32) || !elt_aligned(residual_out, a.res_f32))
    return RSSM_EINVAL;
  a.x = x;
  a.weight = weight;
  a.z = z;
  a.residual = residual;
  a.res_out = residual_out;
  a.out = out;
  a.scale = scale;
  const NormShape sh = norm_shape(a.nvec, false, a.rows);
  if (!grid_fits(a.rows, sh.threads)) return RSSM_ESHAPE;
  const void* fn = f32 ? pick_norm_fwd_kernel<float>(sh) : pick_norm_fwd_kernel<bf16>(sh);
  if (norm_is<1024, 1>(sh))
    fn = f32 ? reinterpret_cast<const void*>(&norm_fwd_kernel<float, 1024, 1>)
             : reinterpret_cast<const void*>(&norm_fwd_kernel<bf16, 1024, 1>);
  return launch_kernel(fn, (unsigned)a.rows, (unsigned)sh.threads, norm_lds(a), stream, a);
}

extern "C" size_t rms_norm_backward_workspace(const rssm_norm_dims* dims) {
  NormArgs a{};
  if (norm_check(dims, &a)) return 0;
  return sizeof(float) * (size_t)bwd_parts(a) * a.dim;
}

extern "C" int rms_norm_backward(const rssm_norm_dims* dims, const void* dy, const void* x,
                                 const float* weight, const void* z, void* dx, float* dweight,
                                 void* dz, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
  NormArgs a{};
  int rc = norm_check(dims, &a);
  if (rc) return rc;
  if (!dweight || !weight) return RSSM_EINVAL;
  if (a.rows > 0 && (!dy || !x || !dx || (z && !dz) || !workspace)) return RSSM_EINVAL;
  const bool f32 = dims->io_dtype == RSSM_F32;
  if (!elt_aligned(x, f32) || !elt_aligned(z, f32) || !elt_aligned(dy, f32) ||
      !elt_aligned(dx, f32) || !elt_aligned(dz, f32))
    return RSSM_EINVAL;
  if (workspace_bytes < rms_norm_backward_workspace(dims)) return RSSM_EINVAL;
  a.dy = dy;
  a.x = x;
  a.weight = weight;
  a.z = z;
  a.dx = dx;
  a.dz = dz;
  a.dweight = dweight;
  a.part = static_cast<float*>(workspace);
  a.parts = bwd_parts(a);
  if (a.rows > 0) {
    const NormShape sh = norm_shape(a.nvec, true);
    const void* fn = f32 ? pick_norm_bwd_kernel<float>(sh) : pick_norm_bwd_kernel<bf16>(sh);
    rc = launch_kernel(fn, (unsigned)a.parts, (unsigned)sh.threads, norm_bwd_lds(a), stream, a);
    if (rc) return rc;
  }
  return launch_kernel(reinterpret_cast<const void*>(&norm_bwd_join_kernel),
                       (unsigned)((a.dim + 15) / 16), 256, 0, stream, a);
}
