// Norm of queries and keys per head with the rotation by position, on gfx950:
//
//   n = x / sqrt(mean(x^2) + eps) w  (RMS),  x / max(||x||, 1e-30)  (L2),  or x
//   out_j = n_j cos t_j - n_j' sin t_j,  out_j' = n_j' cos t_j + n_j sin t_j
//
// for the pairs (j, j') of the first R channels, (j, j + R/2) or (2j, 2j + 1), with the angle
// t_j = position inv_freq_j; the other channels stay n.  Backward, with g the output's
// gradient turned back by the same angle and u = g w:
//   dx = inv (u - x inv^2 share sum(u x)),  share = 1/D (RMS), 1 (L2), 0;  dw = sum_rows g x inv
//
// HBM-bound: every value is read and written once (4 x 4096 tokens of 16 + 8 heads of 128, bf16:
// 201 MB in 52 us, 3.9 TB/s; backward 302 MB in 65 us, 4.7, and 6 for the weights' sums).  A group of lanes holds one row, 16
// bytes a lane; the partner of a channel half a rotation away comes by lane shuffle, as
// loaded.  A workgroup takes one to four tokens with all their heads, so that their angles
// are formed once, in LDS.  An angle of a far position has lost its fraction of a turn in
// fp32 (position 10^6: 0.06 rad), so turns are counted and the quarter taken off in fp64;
// what is left, at most an eighth of a turn, goes through the Taylor sums in fp32.
#include <hip/hip_runtime.h>

#include "gdn_hybrid.h"
#include "gdn_layer_device.h"

namespace gdn {
namespace {

using namespace layer;

// cos and sin of position times frequency (radians).
__device__ __forceinline__ float2 turn_(int32_t pos, float freq) {
  const double turns = static_cast<double>(pos) * static_cast<double>(freq) * 0.15915494309189535;
  const double quarters = rint(4.0 * turns);
  const float x = static_cast<float>((turns - 0.25 * quarters) * 6.283185307179586);  // |x| <= pi / 4
  const int q = static_cast<int>(quarters - 4.0 * floor(0.25 * quarters));
  const float y = x * x;
  // remainders: x^11 / 11! and x^12 / 12!, below 2e-9
  const float s = x * fmaf(y, fmaf(y, fmaf(y, fmaf(y, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), 1.f);
  const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  const float a = (q & 1) ? s : c, b = (q & 1) ? c : s;  // cos and sin but for their signs
  return float2{q == 1 || q == 2 ? -a : a, q >= 2 ? -b : b};
}

// inv and share of a row from its sum of squares.
template <int D>
__device__ __forceinline__ void scale_(int norm, float eps, float ss, float& inv, float& share) {
  inv = 1.f;
  share = 0.f;
  if (norm == GDN_ROPE_RMS) {
    inv = 1.f / sqrtf(ss * (1.f / D) + eps);
    share = 1.f / D;
  } else if (norm == GDN_ROPE_L2) {
    const float n = sqrtf(ss);
    inv = 1.f / (n < 1e-30f ? 1e-30f : n);  // a NaN stays one
    share = n <= 1e-30f ? 0.f : 1.f;
  }
}

template <typename E, int D, bool INTER>
struct Row16 {
  static constexpr int EPV = 16 / static_cast<int>(sizeof(E));  // values of a lane
  static constexpr int LPR = D / EPV;                           // lanes of a row
  static constexpr int RPB = 256 / LPR;                         // rows of a workgroup at a time
};

// The rotation's partner of every value of this lane, as loaded.
template <typename E, int D>
__device__ __forceinline__ Raw<E, 16 / sizeof(E)> partner_(const Raw<E, 16 / sizeof(E)>& v, int sub, int half, int lane) {
  Raw<E, 16 / sizeof(E)> o;
  const int other = sub < half ? lane + half : sub < 2 * half ? lane - half : lane;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.w[0][i] = __shfl(v.w[0][i], other, 64);
  return o;
}

template <typename E, int D, bool INTER, bool BWD>
__global__ __launch_bounds__(256) void rope_kernel(RopeParams p) {
  using S = Row16<E, D, INTER>;
  constexpr int EPV = S::EPV, LPR = S::LPR, RPB = S::RPB;
  const int lane = threadIdx.x & 63, sub = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  const int c0 = sub * EPV, heads = p.Hq + p.Hk, half = p.R / 2;
  __shared__ alignas(16) float cs[kRopeMost][2][D / 2];  // cosines, sines of a token's pairs
  __shared__ alignas(16) float sums[BWD ? RPB : 1][BWD ? D : 4];
  // weights of this lane's channels and of their partners
  const int cp = INTER || c0 >= p.R ? c0 : c0 < half ? c0 + half : c0 - half;
  float w[2][EPV], wp[2][EPV];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float* const ws = k ? p.wk : p.wq;
#pragma unroll
    for (int e = 0; e < EPV; e += 4) {
      const f32x4_t one = {1.f, 1.f, 1.f, 1.f};
      const f32x4_t a = ws ? *reinterpret_cast<const f32x4_t*>(ws + c0 + e) : one, b = ws ? *reinterpret_cast<const f32x4_t*>(ws + cp + e) : one;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[k][e + i] = a[i];
        wp[k][e + i] = b[i];
      }
    }
  }
  float dw[2][EPV];
#pragma unroll
  for (int e = 0; e < EPV; ++e) dw[0][e] = dw[1][e] = 0.f;

  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.per_group; t0 < p.tokens; t0 += static_cast<int64_t>(p.groups) * p.per_group) {
    const int count = static_cast<int>(min(static_cast<int64_t>(p.per_group), p.tokens - t0));
    for (int a = threadIdx.x; a < count * half; a += 256) {
      const int tk = a / half, j = a - tk * half;
      const int32_t pos = p.pos ? p.pos[t0 + tk] : static_cast<int32_t>((t0 + tk) % p.T);
      const float2 t = turn_(pos, p.inv_freq[j]);
      cs[tk][0][j] = t.x;
      cs[tk][1][j] = t.y;
    }
    __syncthreads();
    const int rows = count * heads;
    for (int r0 = 0; r0 < rows; r0 += RPB) {
      const bool live = r0 + slot < rows;
      const int row = live ? r0 + slot : 0, tk = row / heads, h = row - tk * heads;
      const bool key = h >= p.Hq;
      const int64_t token = t0 + tk;
      const E* const src = key ? static_cast<const E*>(p.k) + token * p.k_stride + (h - p.Hq) * D
                               : static_cast<const E*>(p.q) + token * p.q_stride + h * D;
      const int64_t to = key ? (token * p.Hk + (h - p.Hq)) * D + c0 : (token * p.Hq + h) * D + c0;
      Raw<E, EPV> x, d;
      x.load(src + c0);
      if constexpr (BWD) d.load(static_cast<const E*>(key ? p.dk_out : p.dq_out) + to);
      // cosines and sines of this lane's channels; beyond the rotation 1 and 0
      float co[EPV], si[EPV];
#pragma unroll
      for (int e = 0; e < EPV; ++e) {
        const int c = c0 + e;
        const int j = INTER ? c >> 1 : c < half ? c : c - half;
        const bool in = c < p.R;
        co[e] = in ? cs[tk][0][in ? j : 0] : 1.f;
        // the sign with which the partner comes in, forward
        const bool first = INTER ? !(c & 1) : c < half;
        si[e] = in ? (first ? -cs[tk][1][in ? j : 0] : cs[tk][1][in ? j : 0]) : 0.f;
      }
      float inv = 1.f, share = 0.f;
      float ss = 0.f;
      if (BWD || p.norm != GDN_ROPE_NONE) {
#pragma unroll
        for (int e = 0; e < EPV; ++e) ss = fmaf(x.get(e), x.get(e), ss);
#pragma unroll
        for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor(ss, m, 64);
        scale_<D>(p.norm, p.eps, ss, inv, share);
      }
      float out[EPV];
      if constexpr (!BWD) {
        const Raw<E, EPV> xp = INTER ? x : partner_<E, D>(x, sub, half / EPV, lane);
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
          const int o = INTER ? e ^ 1 : e;
          const float n = x.get(e) * inv * (key ? w[1][e] : w[0][e]);
          const float m = xp.get(o) * inv * (INTER ? (key ? w[1][o] : w[0][o]) : (key ? wp[1][e] : wp[0][e]));
          out[e] = c0 + e < p.R ? fmaf(n, co[e], m * si[e]) : n;
        }
      } else {
        const Raw<E, EPV> dp = INTER ? d : partner_<E, D>(d, sub, half / EPV, lane);
        float u[EPV], dot = 0.f;
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
          const int o = INTER ? e ^ 1 : e;
          // turned back: the sines change their signs
          const float g = c0 + e < p.R ? fmaf(d.get(e), co[e], -(dp.get(o) * si[e])) : d.get(e);
          u[e] = g * (key ? w[1][e] : w[0][e]);
          dot = fmaf(u[e], x.get(e), dot);
          const float gx = live ? g * (x.get(e) * inv) : 0.f;
          dw[0][e] += key ? 0.f : gx;
          dw[1][e] += key ? gx : 0.f;
        }
#pragma unroll
        for (int m = 1; m < LPR; m <<= 1) dot += __shfl_xor(dot, m, 64);
        const float along = dot * share * inv * inv;
#pragma unroll
        for (int e = 0; e < EPV; ++e) out[e] = inv * (share > 0.f ? fmaf(-x.get(e), along, u[e]) : u[e]);
      }
      if (live) store_vec<E, EPV>(static_cast<E*>(key ? p.k_out : p.q_out) + to, out);
    }
    __syncthreads();
  }
  if constexpr (BWD) {
    if (!p.dwq && !p.dwk) return;
    // the rows' sums, in order of their places in the workgroup
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int e = 0; e < EPV; ++e) sums[slot][c0 + e] = dw[k][e];
      __syncthreads();
      if (threadIdx.x < D) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < RPB; ++r) s += sums[r][threadIdx.x];
        p.part[(static_cast<int64_t>(blockIdx.x) * 2 + k) * D + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

// The workgroups' sums of 64 channels: each of 16 waves adds every sixteenth in order, then
// the sixteen are added.
__global__ __launch_bounds__(1024) void rope_weight_kernel(RopeParams p, int D) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, at = blockIdx.x * 64 + lane;  // at: of 2 D
  __shared__ float part[16][64];
  float s = 0.f;
#pragma unroll 8
  for (int g = wave; g < p.groups; g += 16) s += p.part[static_cast<int64_t>(g) * 2 * D + at];
  part[wave][lane] = s;
  __syncthreads();
  if (wave) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += part[i][lane];
  float* const out = at < D ? p.dwq : p.dwk;
  if (out) out[at < D ? at : at - D] = s;
}

template <typename E, int D, bool BWD>
hipError_t launch_d(const RopeParams& p, bool interleaved, hipStream_t s) {
  if (p.groups > 0) {
    if (interleaved)
      hipLaunchKernelGGL((rope_kernel<E, D, true, BWD>), dim3(static_cast<unsigned>(p.groups)), dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((rope_kernel<E, D, false, BWD>), dim3(static_cast<unsigned>(p.groups)), dim3(256), 0, s, p);
  }
  if (BWD && (p.dwq || p.dwk)) hipLaunchKernelGGL(rope_weight_kernel, dim3(2 * D / 64), dim3(1024), 0, s, p, D);
  return hipGetLastError();
}

template <typename E, bool BWD>
hipError_t launch_e(const RopeParams& p, int D, bool interleaved, hipStream_t s) {
  switch (D) {
    case 64: return launch_d<E, 64, BWD>(p, interleaved, s);
    case 128: return launch_d<E, 128, BWD>(p, interleaved, s);
    case 256: return launch_d<E, 256, BWD>(p, interleaved, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_rope_fwd(const RopeParams& p, int D, bool bf16, bool interleaved, hipStream_t s) {
  return bf16 ? launch_e<uint16_t, false>(p, D, interleaved, s) : launch_e<float, false>(p, D, interleaved, s);
}

hipError_t launch_rope_bwd(const RopeParams& p, int D, bool bf16, bool interleaved, hipStream_t s) {
  return bf16 ? launch_e<uint16_t, true>(p, D, interleaved, s) : launch_e<float, true>(p, D, interleaved, s);
}

}  // namespace gdn
