// One token of the gated delta rule for every (sequence, head) on gfx950, scalar or
// per-key-channel decay, state updated in place:
//     S <- exp(g) S;  e = beta (v - S^T k);  S <- S + k e^T;  o = scale S^T q
//
// The two column sums r = S'^T k and s = S'^T q of the decayed state S' = exp(g) S
// come from one pass over it, and o = scale (s + (k . q) e) needs no second one, so
// the state is read and written once: the work is HBM-bound (2 Dk Dv fp32 against
// about 7 Dk Dv operations).
//
// A workgroup holds Dk rows of COLS columns of one state in registers (lanes of four
// columns, the rows of a thread 1024 / COLS apart); neighbouring workgroups hold
// neighbouring columns.  All products are fp32.  Measured, Dk = Dv = 128, bf16:
//   128 x 16 heads (271 MB): 47.6 us, 5.7 TB/s, with 64 columns and streaming accesses;
//   60 us with 32 columns and cached ones (51 with the first change alone, 59 with the second);
//   8 heads (1 MB): 3.8 us with 32 columns (32 workgroups), 4.0 with 64.
#include <hip/hip_runtime.h>

#include "gdn_chunk_common.h"
#include "gdn_device.h"
#include "gdn_layer.h"

namespace gdn {
namespace {

// STREAM: the states are read and written past the caches.
template <typename E, int DK, bool CHAN, int COLS, bool STREAM>
__global__ __launch_bounds__(256) void step_kernel(StepParams p) {
  constexpr int CL = COLS / 4;   // lanes of a row
  constexpr int RG = 256 / CL;   // rows at a time
  constexpr int R = DK / RG;     // rows of a thread
  const int tid = threadIdx.x, cl = tid % CL, row0 = tid / CL;
  const int tiles = (p.Dv + COLS - 1) / COLS;
  const int64_t head = blockIdx.x / tiles;
  const int col = (blockIdx.x % tiles) * COLS + cl * 4;
  const bool live = col < p.Dv;
  float* const S = p.S + head * DK * p.Dv + col;
  const E* const qp = static_cast<const E*>(p.q) + head * DK;
  const E* const kp = static_cast<const E*>(p.k) + head * DK;

  f32x4_t s[R];
  float kf[R], qf[R], a[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + RG * r;
    const f32x4_t* const at = reinterpret_cast<const f32x4_t*>(S + static_cast<int64_t>(row) * p.Dv);
    s[r] = !live ? zero4() : STREAM ? __builtin_nontemporal_load(at) : *at;
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
  // over the row groups of the wave, then over the four waves
#pragma unroll
  for (int m = CL; m < 64; m <<= 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sk[j] += __shfl_xor(sk[j], m, 64);
      sq[j] += __shfl_xor(sq[j], m, 64);
    }
    kq += __shfl_xor(kq, m, 64);
  }
  __shared__ float red[4][CL][9];
  const int wave = tid >> 6, lane = tid & 63;
  if (lane < CL) {
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
    f32x4_t* const at = reinterpret_cast<f32x4_t*>(S + static_cast<int64_t>(row0 + RG * r) * p.Dv);
    if (STREAM)
      __builtin_nontemporal_store(s[r], at);
    else
      *at = s[r];
  }
  if (row0 == 0) {
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = p.scale * fmaf(t[8], e[j], t[4 + j]);
    chunk::store4<E>(static_cast<E*>(p.o) + head * p.Dv + col, o[0], o[1], o[2], o[3]);
  }
}

template <typename E, int DK, bool CHAN>
hipError_t launch_t(const StepParams& p, hipStream_t s) {
  // states that the L2 caches (32 MB) hold between two tokens stay there
  if (p.heads * DK * p.Dv * 4 < (32 << 20)) {
    const int64_t tiles = (p.Dv + 31) / 32;
    hipLaunchKernelGGL((step_kernel<E, DK, CHAN, 32, false>), dim3(static_cast<unsigned>(p.heads * tiles)), dim3(256), 0, s, p);
  } else {
    const int64_t tiles = (p.Dv + 63) / 64;
    hipLaunchKernelGGL((step_kernel<E, DK, CHAN, 64, true>), dim3(static_cast<unsigned>(p.heads * tiles)), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

template <typename E>
hipError_t launch_e(const StepParams& p, int Dk, bool channel, hipStream_t s) {
  if (Dk == 64) return channel ? launch_t<E, 64, true>(p, s) : launch_t<E, 64, false>(p, s);
  return channel ? launch_t<E, 128, true>(p, s) : launch_t<E, 128, false>(p, s);
}

}  // namespace

hipError_t launch_step(const StepParams& p, int Dk, bool bf16, bool channel, hipStream_t s) {
  return bf16 ? launch_e<uint16_t>(p, Dk, channel, s) : launch_e<float>(p, Dk, channel, s);
}

}  // namespace gdn
