// One token of linear attention for a batch of rows: S = g S + v k^T, o = scale S q.
//
// Memory bound: every state is read and written once (8 K V bytes for 5 K V
// operations).  A workgroup takes one row and value head, 16 vectors of four state
// elements a thread (8 where K or V is 64, 4 where both are), all of them in flight
// before the first is used; the lanes of a state row add up o by a transposing butterfly.  256 rows of 32
// heads of 128 x 128: 1.07 GB in 187 us, 5.8 TB/s (a large copy on this card 4.7 to 5.1).
#include "mixer_common.hpp"

namespace rssm {

struct StepArgs {
  MixArgs m;
  const float* state;
  float* new_state;
};

template <typename T, int V, int K>
__global__ void __launch_bounds__(256) mix_step_kernel(const StepArgs s) {
  constexpr int LPR = K / 4, NT = 256, RPI = NT / LPR, ITEMS = V / RPI;
  typedef RowReduce<ITEMS, LPR> Red;
  const MixArgs& a = s.m;
  const int id = xcd_tile(blockIdx.x, gridDim.x);
  const int b = id / a.v_heads, hv = id % a.v_heads, hk = hv / a.vpk;
  const int tid = threadIdx.x, lane = tid & 63, c = (tid % LPR) * 4, row = tid / LPR;
  const int slot = mix_slot(a, b);
  if (slot < 0) {
    if (tid == 0 && hv == 0 && a.status) atomicOr(a.status, RSSM_ST_BAD_SLOT);
    if (tid < V) Elt<T>::store1(a.o, ((long)b * a.v_heads + hv) * V + tid, __int_as_float(0x7fc00000));
    return;
  }
  const long base = ((long)slot * a.v_heads + hv) * (V * K);
  u32x4 raw[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) raw[i] = ld16_stream(s.state, (base + (long)(i * RPI + row) * K + c) * 4);
  float k4[4], q4[4], v[ITEMS];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    k4[e] = Elt<T>::load1(a.k, b * a.k_stride + (long)hk * K + c + e);
    q4[e] = Elt<T>::load1(a.q, b * a.q_stride + (long)hk * K + c + e);
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) v[i] = Elt<T>::load1(a.v, b * a.v_stride + (long)hv * V + i * RPI + row);
  const float decay = a.decay ? expf(a.decay == RSSM_DECAY_HEAD ? a.g[hv] : a.g[(long)b * a.v_heads + hv]) : 1.f;
  float o[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    float f[4];
    Elt<float>::unpack(raw[i], f);
    o[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = fmaf(v[i], k4[e], decay * f[e]);
      o[i] = fmaf(f[e], q4[e], o[i]);
    }
    st16_stream(s.new_state, (base + (long)(i * RPI + row) * K + c) * 4, Elt<float>::pack(f));
  }
  Red::run(o, lane);
  if (Red::DUP == 1 || (lane & (Red::DUP - 1)) == 0) {
#pragma unroll
    for (int j = 0; j < Red::NF; ++j)
      Elt<T>::store1(a.o, ((long)b * a.v_heads + hv) * V + Red::item(j, lane) * RPI + row, a.scale * o[j]);
  }
}

template <typename T>
static const void* pick_step(int dk, int dv) {
  if (dk == 64)
    return dv == 64 ? reinterpret_cast<const void*>(&mix_step_kernel<T, 64, 64>)
                    : reinterpret_cast<const void*>(&mix_step_kernel<T, 128, 64>);
  return dv == 64 ? reinterpret_cast<const void*>(&mix_step_kernel<T, 64, 128>)
                  : reinterpret_cast<const void*>(&mix_step_kernel<T, 128, 128>);
}

}  // namespace rssm

using namespace rssm;

extern "C" int linear_attention_decode(const rssm_mixer_dims* dims, const float* state,
                                       const int32_t* slot_idx, const void* q, const void* k,
                                       const void* v, const float* log_decay, float* new_state, void* o,
                                       int32_t* status, hipStream_t stream) {
  const int rc = mix_check(dims, false);
  if (rc) return rc;
  const rssm_mixer_dims& d = *dims;
  if (d.tokens == 0) return RSSM_OK;
  if (!state || !new_state || !q || !k || !v || !o || (d.decay && !log_decay)) return RSSM_EINVAL;
  if (!aligned16(state) || !aligned16(new_state)) return RSSM_EINVAL;
  StepArgs s{};
  s.m.q = q;
  s.m.k = k;
  s.m.v = v;
  s.m.g = log_decay;
  s.m.slot_idx = slot_idx;
  s.m.o = o;
  s.m.status = status;
  s.state = state;
  s.new_state = new_state;
  mix_fill(s.m, d);
  const long grid = (long)d.tokens * d.v_heads;
  if (!grid_fits(grid, 256)) return RSSM_ESHAPE;
  if (output_meets(s.m, d, o) || pools_meet(d, state, new_state)) return RSSM_EINVAL;
  const void* fn = d.io_dtype == RSSM_F32 ? pick_step<float>(d.dk, d.dv) : pick_step<bf16>(d.dk, d.dv);
  return launch_kernel(fn, (unsigned)grid, 256, 0, stream, s);
}
