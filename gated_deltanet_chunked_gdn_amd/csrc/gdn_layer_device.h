// Device helpers shared by the convolution and scan kernels: rows of 16 bytes as
// fp32 values, and the gate functions in fp32.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_chunk_common.h"
#include "gdn_device.h"

namespace gdn {
namespace layer {

using chunk::u32x4_t;
constexpr float kLog2e = chunk::kLog2e;

// NV elements of type E held as loaded (vectors of 16 bytes, or one of 8), and as
// fp32.
template <typename E, int NV>
struct Raw {
  static constexpr int kBytes = NV * static_cast<int>(sizeof(E));
  static constexpr int kLanes = kBytes >= 16 ? 4 : 2;  // dwords of a vector
  static constexpr int kVecs = kBytes / (4 * kLanes);
  static_assert(kVecs * kLanes * 4 == kBytes, "whole vectors");
  typedef uint32_t vec_t __attribute__((ext_vector_type(kLanes)));
  vec_t w[kVecs];
  __device__ __forceinline__ void load(const E* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) w[i] = reinterpret_cast<const vec_t*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) w[i] = vec_t(0u);
  }
  __device__ __forceinline__ float get(int e) const {
    const int word = sizeof(E) == 2 ? e >> 1 : e;
    const uint32_t x = w[word / kLanes][word % kLanes];
    if constexpr (sizeof(E) == 2)
      return __uint_as_float((e & 1) ? (x & 0xffff0000u) : (x << 16));
    else
      return __uint_as_float(x);
  }
};

// NV fp32 values rounded once and stored as vectors of 16 bytes, or one of 8.
template <typename E, int NV>
__device__ __forceinline__ void store_vec(E* p, const float* f) {
  if constexpr (sizeof(E) == 2 && NV == 4) {
    *reinterpret_cast<uint2*>(p) = uint2{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
  } else if constexpr (sizeof(E) == 2) {
#pragma unroll
    for (int i = 0; i < NV / 8; ++i)
      reinterpret_cast<u32x4_t*>(p)[i] = u32x4_t{pack_bf16x2(f[8 * i], f[8 * i + 1]), pack_bf16x2(f[8 * i + 2], f[8 * i + 3]),
                                                 pack_bf16x2(f[8 * i + 4], f[8 * i + 5]), pack_bf16x2(f[8 * i + 6], f[8 * i + 7])};
  } else {
#pragma unroll
    for (int i = 0; i < NV / 4; ++i)
      reinterpret_cast<u32x4_t*>(p)[i] = u32x4_t{__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                                 __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3])};
  }
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_(float x) { return __builtin_amdgcn_rcpf(x); }
// 1 / (1 + exp(-x)); 0 and 1 at the infinities
__device__ __forceinline__ float sigmoid_(float x) { return rcp_(1.f + exp2_(-kLog2e * x)); }

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1].  With w = 1 + e rounded,
// log1p(e) = log(w) + (e - (w - 1)) / w up to the square of the second term, the
// rounding of w, r = |e - (w - 1)| <= 2^-24 (w lies in [1, 2]).  Dividing it by w is left
// out, which adds r (w - 1) / w.  On [1, 2] log(w) >= (w - 1) log 2, so where w > 1 that is
// at most r / (w log 2) <= 1.45 2^-24 of the logarithm; where w == 1 nothing is added and
// the sum is e itself.  `sig` gets the derivative, sigmoid(x).
__device__ __forceinline__ float softplus_(float x, float& sig) {
  const float e = exp2_(-kLog2e * fabsf(x)), w = 1.f + e;
  const float r = rcp_(w);
  sig = x >= 0.f ? r : e * r;
  const float l = fmaf(__builtin_amdgcn_logf(w), 0.6931471805599453f, e - (w - 1.f));
  return l + fmaxf(x, 0.f);
}

// The sequence that holds packed row t: the last n with cu[n] <= t.
__device__ __forceinline__ int seq_of_row(const SeqInfo& s, int N, int64_t t) {
  if (!s.cu) return static_cast<int>(t / s.T);
  int lo = 0, hi = N;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.cu[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

}  // namespace layer
}  // namespace gdn
