// One token of the gated delta rule for every (sequence, head) on gfx950, scalar or
// per-key-channel decay, state updated in place:
//     S <- exp(g) S;  e = beta (v - S^T k);  S <- S + k e^T;  o = scale S^T q
//
// The two column sums r = S'^T k and s = S'^T q of the decayed state S' = exp(g) S
// come from one pass over it, and o = scale (s + (k . q) e) needs no second one, so
// the state is read and written once: the work is HBM-bound (2 Dk Dv fp32 against
// about 7 Dk Dv operations).
//
// A workgroup holds Dk rows x 32 columns of one state in registers (eight lanes of
// four columns a row, 128-byte row pieces; a thread's rows are 32 apart), so that a
// few heads still spread over the chip.  All products are fp32.
#include <hip/hip_runtime.h>

#include "gdn_chunk_common.h"
#include "gdn_device.h"
#include "gdn_layer.h"

namespace gdn {
namespace {

constexpr int kCols = 32;  // state columns of a workgroup

template <typename E, int DK, bool CHAN>
__global__ __launch_bounds__(256) void step_kernel(StepParams p) {
  constexpr int R = DK / 32;  // rows of a thread
  const int tid = threadIdx.x, cl = tid & 7, row0 = tid >> 3;
  const int64_t head = blockIdx.x;
  const int col = blockIdx.y * kCols + cl * 4;
  const bool live = col < p.Dv;
  float* const S = p.S + head * DK * p.Dv + col;
  const E* const qp = static_cast<const E*>(p.q) + head * DK;
  const E* const kp = static_cast<const E*>(p.k) + head * DK;

  f32x4_t s[R];
  float kf[R], qf[R], a[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + 32 * r;
    s[r] = live ? *reinterpret_cast<const f32x4_t*>(S + static_cast<int64_t>(row) * p.Dv) : zero4();
    kf[r] = IoT<E>::ld(kp + row);
    qf[r] = IoT<E>::ld(qp + row);
    a[r] = CHAN ? p.g[head * DK + row] : p.g[head];
  }
  const float beta = p.beta[head];
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = live ? IoT<E>::ld(static_cast<const E*>(p.v) + head * p.Dv + col + j) : 0.f;

  f32x4_t sk = zero4(), sq = zero4();
  float kq = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float d = expf(a[r]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[r][j] *= d;
      sk[j] = fmaf(s[r][j], kf[r], sk[j]);
      sq[j] = fmaf(s[r][j], qf[r], sq[j]);
    }
    kq = fmaf(kf[r], qf[r], kq);
  }
  // over the eight row groups of the wave, then over the four waves
#pragma unroll
  for (int m = 8; m < 64; m <<= 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sk[j] += __shfl_xor(sk[j], m, 64);
      sq[j] += __shfl_xor(sq[j], m, 64);
    }
    kq += __shfl_xor(kq, m, 64);
  }
  __shared__ float red[4][8][9];
  const int wave = tid >> 6, lane = tid & 63;
  if (lane < 8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      red[wave][lane][j] = sk[j];
      red[wave][lane][4 + j] = sq[j];
    }
    red[wave][lane][8] = kq;
  }
  __syncthreads();
  float t[9];
#pragma unroll
  for (int j = 0; j < 9; ++j) t[j] = (red[0][cl][j] + red[1][cl][j]) + (red[2][cl][j] + red[3][cl][j]);
  float e[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) e[j] = beta * (v[j] - t[j]);
  if (!live) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s[r][j] = fmaf(kf[r], e[j], s[r][j]);
    *reinterpret_cast<f32x4_t*>(S + static_cast<int64_t>(row0 + 32 * r) * p.Dv) = s[r];
  }
  if (row0 == 0) {
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = p.scale * fmaf(t[8], e[j], t[4 + j]);
    chunk::store4<E>(static_cast<E*>(p.o) + head * p.Dv + col, o[0], o[1], o[2], o[3]);
  }
}

template <typename E, int DK>
hipError_t launch_t(const StepParams& p, bool channel, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.heads), static_cast<unsigned>((p.Dv + kCols - 1) / kCols));
  if (channel)
    hipLaunchKernelGGL((step_kernel<E, DK, true>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((step_kernel<E, DK, false>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_step(const StepParams& p, int Dk, bool bf16, bool channel, hipStream_t s) {
  if (Dk == 64) return bf16 ? launch_t<uint16_t, 64>(p, channel, s) : launch_t<float, 64>(p, channel, s);
  return bf16 ? launch_t<uint16_t, 128>(p, channel, s) : launch_t<float, 128>(p, channel, s);
}

}  // namespace gdn
