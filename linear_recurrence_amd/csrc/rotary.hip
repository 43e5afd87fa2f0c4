// Rotary positions: pairs of a head's elements turned by position * frequency.
//
// Memory bound: each element is read and written once.  A workgroup takes a few
// tokens and a range of heads.  First a thread for each (token, pair) forms the
// angle in turns, its fraction, sine and cosine in double (at position 2^20 an fp32
// angle would be off by 0.06), once for all heads; then a thread keeps the sines of
// its pairs of one token in registers and walks the heads with two loads on their way.
// Elements that only pass take the same way, so that lanes that turn and lanes that copy
// load together.
// 16383 tokens of 64 heads of 128: 109 us, 4.9 TB/s; 8192 of 48 heads, half of each
// interleaved: a call among others 44 us, 4.6 TB/s (63 with the copying lanes in a branch of
// their own), and the kernel alone, on the same inputs in a row, 32.
#include <math.h>

#include "rssm_host.hpp"
#include "seq_device.hpp"

namespace rssm {

struct RotaryArgs {
  const void* x;
  const void* pos;
  const float* freqs;
  void* y;
  long x_stride, y_stride;
  int32_t tokens, heads, dim, half, interleaved, pos_int64, inverse;
  int32_t tok, hpg, groups;  // tokens a workgroup, heads a group, groups of heads
  int32_t turn, items;       // a head's items of pairs; those and the items of copied elements
  float amplitude;
};

constexpr int kRotTable = 512;  // (token, pair) entries of a workgroup

template <typename T, bool INTER>
__global__ void __launch_bounds__(256) rotary_kernel(const RotaryArgs a) {
  __shared__ float2 sT[kRotTable];
  const int tid = threadIdx.x;
  const int blk = blockIdx.x / a.groups, h0 = (blockIdx.x % a.groups) * a.hpg;
  const int h1 = h0 + a.hpg < a.heads ? h0 + a.hpg : a.heads;
  const long t0 = (long)blk * a.tok;
  const int toks = a.tokens - t0 < a.tok ? (int)(a.tokens - t0) : a.tok;
  for (int e = tid; e < toks * a.half; e += 256) {
    const int t = e / a.half, i = e - t * a.half;
    const double p = a.pos_int64 ? (double)static_cast<const int64_t*>(a.pos)[t0 + t]
                                 : (double)static_cast<const int32_t*>(a.pos)[t0 + t];
    const double turns = p * (double)a.freqs[i] * 0.15915494309189533577;
    double s, c;
    sincospi(2.0 * (turns - rint(turns)), &s, &c);
    const double amp = a.amplitude;
    sT[e] = make_float2((float)(amp * c), (float)(a.inverse ? -amp * s : amp * s));
  }
  __syncthreads();
  // A thread's item: one vector of 8 elements (INTER: 4 pairs, or copies), or two (8 pairs,
  // one element of each in either; or copies).
  constexpr int NV = INTER ? 1 : 2, NP = INTER ? 4 : 8, U = 2 / NV;
  const int step = 256 / a.items, hh = tid / a.items, it = tid - hh * a.items;
  if (hh >= step) return;
  const bool turns = it < a.turn;
  int off[NV], n[NV];
  const int i0 = NP * it;  // the first pair
  if (turns) {
    const int m = a.half - i0 < NP ? a.half - i0 : NP;
    off[0] = INTER ? 2 * i0 : i0;
    n[0] = INTER ? 2 * m : m;
    if (!INTER) off[NV - 1] = a.half + i0, n[NV - 1] = m;
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      off[v] = 2 * a.half + 8 * (NV * (it - a.turn) + v);
      n[v] = a.dim - off[v] < 0 ? 0 : (a.dim - off[v] < 8 ? a.dim - off[v] : 8);
    }
  }
  for (int t = 0; t < toks; ++t) {
    const long xr = (t0 + t) * a.x_stride, yr = (t0 + t) * a.y_stride;
    float co[NP], si[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const float2 w = turns && i0 + k < a.half ? sT[t * a.half + i0 + k] : make_float2(0.f, 0.f);
      co[k] = w.x;
      si[k] = w.y;
    }
    const auto load = [&](int h, float (*f)[8]) {
#pragma unroll
      for (int v = 0; v < NV; ++v) load8<T>(a.x, xr + (long)h * a.dim + off[v], n[v], f[v]);
    };
    const auto finish = [&](int h, float (*f)[8]) {
      if (turns) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          float& x0 = INTER ? f[0][2 * k] : f[0][k];
          float& x1 = INTER ? f[0][2 * k + 1] : f[NV - 1][k];
          const float p0 = x0, p1 = x1;
          x0 = fmaf(p0, co[k], -p1 * si[k]);
          x1 = fmaf(p0, si[k], p1 * co[k]);
        }
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) store8<T>(a.y, yr + (long)h * a.dim + off[v], n[v], f[v]);
    };
    int h = h0 + hh;
    float f[U][NV][8];
    for (; h + (U - 1) * step < h1; h += U * step) {
#pragma unroll
      for (int u = 0; u < U; ++u) load(h + u * step, f[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) finish(h + u * step, f[u]);
    }
    if (U > 1 && h < h1) {
      load(h, f[0]);
      finish(h, f[0]);
    }
  }
}

// Whether rows of x and y share memory.  Two slices of the same wider rows do not.
static bool rotary_overlap(const void* x, long xs, const void* y, long ys, long rows, long row, long es) {
  const char* const px = static_cast<const char*>(x);
  const char* const py = static_cast<const char*>(y);
  if (xs == ys) {
    const long off = ((py - px) % (xs * es) + xs * es) % (xs * es);
    if (off >= row * es && off <= (xs - row) * es) return false;
  }
  return px < py + ((rows - 1) * ys + row) * es && py < px + ((rows - 1) * xs + row) * es;
}

static int rotary(const rssm_rotary_dims* dims, const void* x, const void* positions, const float* freqs,
                  void* y, bool inverse, hipStream_t stream) {
  if (!dims) return RSSM_EINVAL;
  const rssm_rotary_dims& d = *dims;
  if (d.tokens < 0 || d.heads < 1 || d.dim < 2 || d.rotary_dim < 2 || d.rotary_dim > d.dim || d.rotary_dim % 2)
    return RSSM_EINVAL;
  if (!valid_dtype(d.io_dtype)) return RSSM_EDTYPE;
  // a thread's head, and the one that it steps to, are counted in 32 bits
  if (d.dim > 1024 || d.heads > 1 << 30) return RSSM_ESHAPE;
  const long row = (long)d.heads * d.dim, es = d.io_dtype == RSSM_F32 ? 4 : 2;
  if ((d.x_stride && d.x_stride < row) || (d.y_stride && d.y_stride < row)) return RSSM_EINVAL;
  if (d.tokens == 0) return RSSM_OK;
  if (!x || !positions || !freqs || !y) return RSSM_EINVAL;
  if (reinterpret_cast<uintptr_t>(x) % es || reinterpret_cast<uintptr_t>(y) % es ||
      reinterpret_cast<uintptr_t>(positions) % (d.pos_int64 ? 8 : 4))
    return RSSM_EINVAL;
  RotaryArgs a{};
  a.x = x;
  a.pos = positions;
  a.freqs = freqs;
  a.y = y;
  a.x_stride = d.x_stride ? d.x_stride : row;
  a.y_stride = d.y_stride ? d.y_stride : row;
  const bool same = x == y && a.x_stride == a.y_stride;
  if (!same && rotary_overlap(x, a.x_stride, y, a.y_stride, d.tokens, row, es)) return RSSM_EINVAL;
  a.tokens = d.tokens;
  a.heads = d.heads;
  a.dim = d.dim;
  a.half = d.rotary_dim / 2;
  a.interleaved = d.interleaved;
  a.pos_int64 = d.pos_int64;
  a.inverse = inverse;
  a.amplitude = d.amplitude;
  const int rest = same ? 0 : d.dim - d.rotary_dim;
  a.turn = d.interleaved ? (a.half + 3) / 4 : (a.half + 7) / 8;
  a.items = a.turn + (d.interleaved ? (rest + 7) / 8 : (rest + 15) / 16);
  // Tokens enough for a thread each in the table, while there are 1024 workgroups;
  // then the heads are split until there are, down to one round of the threads.
  a.tok = 256 / a.half < 1 ? 1 : 256 / a.half;
  while (a.tok > 1 && ((long)d.tokens + a.tok - 1) / a.tok < 1024) a.tok = (a.tok + 1) / 2;
  const long blocks = ((long)d.tokens + a.tok - 1) / a.tok;
  const int step = 256 / a.items;
  a.hpg = d.heads;
  while (a.hpg > step && blocks * ((d.heads + a.hpg - 1) / a.hpg) < 1024) a.hpg = (a.hpg + 1) / 2;
  a.groups = (d.heads + a.hpg - 1) / a.hpg;
  const long grid = blocks * a.groups;
  if (!grid_fits(grid, 256)) return RSSM_ESHAPE;
  const void* fn = d.io_dtype == RSSM_F32
      ? (d.interleaved ? reinterpret_cast<const void*>(&rotary_kernel<float, true>)
                       : reinterpret_cast<const void*>(&rotary_kernel<float, false>))
      : (d.interleaved ? reinterpret_cast<const void*>(&rotary_kernel<bf16, true>)
                       : reinterpret_cast<const void*>(&rotary_kernel<bf16, false>));
  return launch_kernel(fn, (unsigned)grid, 256, 0, stream, a);
}

}  // namespace rssm

extern "C" int rotary_forward(const rssm_rotary_dims* dims, const void* x, const void* positions,
                              const float* freqs, void* y, hipStream_t stream) {
  return rssm::rotary(dims, x, positions, freqs, y, false, stream);
}

extern "C" int rotary_backward(const rssm_rotary_dims* dims, const void* dy, const void* positions,
                               const float* freqs, void* dx, hipStream_t stream) {
  return rssm::rotary(dims, dy, positions, freqs, dx, true, stream);
}
