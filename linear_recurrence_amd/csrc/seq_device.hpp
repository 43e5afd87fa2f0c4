// Device helpers of the sequence operators (scan, short convolution, norm).
#pragma once

#include <type_traits>

#include "rssm_device.hpp"
#include "seq_index.hpp"

namespace rssm {

// Sixteen bytes at any element boundary: rows of odd length start anywhere.
// gfx950 does such a load or store in one instruction.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

// Two fp32 -> packed bf16, round to nearest even, in one instruction.
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ static inline uint32_t bf16_pk(float lo, float hi) {
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
}

// Eight consecutive elements as fp32.
template <typename T> struct Vec8;

template <> struct Vec8<float> {
  __device__ static inline void load(const void* p, long i, float* f) {
    const float* q = static_cast<const float*>(p) + i;
    const u32x4 a = *reinterpret_cast<const u32x4_any*>(q);
    const u32x4 b = *reinterpret_cast<const u32x4_any*>(q + 4);
    Elt<float>::unpack(a, f);
    Elt<float>::unpack(b, f + 4);
  }
  __device__ static inline void store(void* p, long i, const float* f) {
    float* q = static_cast<float*>(p) + i;
    *reinterpret_cast<u32x4_any*>(q) = Elt<float>::pack(f);
    *reinterpret_cast<u32x4_any*>(q + 4) = Elt<float>::pack(f + 4);
  }
};

template <> struct Vec8<bf16> {
  __device__ static inline void load(const void* p, long i, float* f) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    const u32x4 v = *reinterpret_cast<const u32x4_any*>(q);
    Elt<bf16>::unpack(v, f);
  }
  __device__ static inline void store(void* p, long i, const float* f) {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    const u32x4 v = {bf16_pk(f[0], f[1]), bf16_pk(f[2], f[3]), bf16_pk(f[4], f[5]),
                     bf16_pk(f[6], f[7])};
    *reinterpret_cast<u32x4_any*>(q) = v;
  }
};

// The first n (0..8) of eight consecutive elements; the others read as 0.
template <typename T>
__device__ static inline void load8(const void* p, long i, int n, float* f) {
  if (n == 8) {
    Vec8<T>::load(p, i, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = k < n ? Elt<T>::load1(p, i + k) : 0.f;
  }
}
template <typename T>
__device__ static inline void store8(void* p, long i, int n, const float* f) {
  if (n == 8) {
    Vec8<T>::store(p, i, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) Elt<T>::store1(p, i + k, f[k]);
  }
}

// K consecutive elements (8 or 4) as they are stored.
template <typename T, int K>
struct RawK {
  static constexpr int kWords = K * (sizeof(T) == 4 ? 4 : 2) / 8;  // pairs of 32 bits
  u32x2 v[kWords];
  __device__ inline void zero() {
#pragma unroll
    for (int q = 0; q < kWords; ++q) v[q] = u32x2{0, 0};
  }
  // the first n of them, the others 0
  __device__ inline void load(const void* p, long i, int n) {
    typedef typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type E;
    const E* const q = static_cast<const E*>(p) + i;
    if (n == K) {
      if constexpr (kWords == 1) {
        v[0] = *reinterpret_cast<const u32x2_any*>(q);
      } else {
#pragma unroll
        for (int w = 0; w < kWords; w += 2) {
          const u32x4 x = *reinterpret_cast<const u32x4_any*>(q + w * (8 / sizeof(E)));
          v[w] = u32x2{x[0], x[1]};
          v[w + 1] = u32x2{x[2], x[3]};
        }
      }
    } else {
      constexpr int kPer = 4 / sizeof(E);
#pragma unroll
      for (int w = 0; w < 2 * kWords; ++w) {
        uint32_t x = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (w * kPer + k < n) x |= (uint32_t)q[w * kPer + k] << (16 * k);
        v[w >> 1][w & 1] = x;
      }
    }
  }
  __device__ inline void get(float* f) const {
#pragma unroll
    for (int w = 0; w < 2 * kWords; ++w) {
      const uint32_t x = v[w >> 1][w & 1];
      if constexpr (sizeof(T) == 4) {
        f[w] = __uint_as_float(x);
      } else {
        f[2 * w] = __uint_as_float(x << 16);
        f[2 * w + 1] = __uint_as_float(x & 0xffff0000u);
      }
    }
  }
};
template <typename T, int K>
__device__ static inline void store_k(void* p, long i, int n, const float* f) {
  if constexpr (K == 8) {
    store8<T>(p, i, n, f);
  } else if (n < K) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < n) Elt<T>::store1(p, i + k, f[k]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<u32x4_any*>(static_cast<float*>(p) + i) = Elt<float>::pack(f);
  } else {
    *reinterpret_cast<u32x2_any*>(static_cast<uint16_t*>(p) + i) = u32x2{bf16_pk(f[0], f[1]), bf16_pk(f[2], f[3])};
  }
}

// sigmoid(v) = 1 / (1 + e^-v); e^-v overflows to Inf below -88, where the
// quotient is the correct 0.  Hardware exp and reciprocal (about 2 ulp).
__device__ static inline float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-v));
}

// softplus(v) = log(1 + e^v): v itself above 20 (exact in fp32).  The library's
// log1p rather than softplus_f32's hardware log: near 1 that one is off by more
// than an ulp of the logarithm, which the sums over tokens of the decay's
// gradient would carry whole.
__device__ static inline float softplus_exact(float v) { return v > 20.f ? v : log1pf(expf(v)); }

// All of the table, by one workgroup: a kernel whose work is found by searching
// the table does not meet every entry of one that is not monotone.
__device__ static inline void check_table(const int32_t* cu, int nseq, int tokens, int32_t* status) {
  if (!cu || !status) return;
  bool bad = false;
  for (int i = threadIdx.x; i < nseq; i += blockDim.x) bad |= seq_span(cu, i, nseq, tokens).bad;
  if (bad) atomicOr(status, RSSM_ST_BAD_SEQ);
}

}  // namespace rssm
