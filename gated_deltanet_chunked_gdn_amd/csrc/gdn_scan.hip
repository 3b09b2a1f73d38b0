// Selective state space scan on gfx950: forward (serial or split over the time axis)
// and the single-token step.
//     delta = softplus(dt + bias);  h <- exp(delta A) h + delta u B;  s = C . h + D u
// per channel, with N states a channel; y = s, or s silu(z).
//
// What bounds it: per token, channel and state one multiply and one exponential for
// the decay, one multiply for the write, two fused multiply-adds for the state and
// the output -- vector instructions, all in fp32, against N / (a few) bytes of HBM
// traffic.  So the layout keeps everything else out of the inner loop:
//   * four lanes share a channel, each holding N / 4 of its states in registers; the
//     states of one lane are contiguous, so B and C come from LDS as wide reads that
//     sixteen channels share;
//   * a workgroup of four waves (64 channels) stages a tile of 16 tokens: delta and
//     delta u are formed once per (token, channel), the softplus with them;
//   * the four partial outputs of a channel are reduced for four tokens at a time by
//     two lane swaps (v_permlane32_swap, v_permlane16_swap): three swaps and three
//     adds leave each of the four lanes with one token's sum;
//   * the next tile's global loads are in flight while a tile is computed, and the
//     outputs leave through LDS as 16-byte row pieces.
#include <hip/hip_runtime.h>

#include "gdn_scan_device.h"

namespace gdn {
namespace {

using namespace layer;
using namespace scan;

// kSummary: end state from a zero start and the sum of delta of every segment but a
// sequence's last; kFull: outputs, from the composed start.
enum Mode { kSummary, kFull };

template <typename E, int N, Mode M>
__global__ __launch_bounds__(256) void scan_fwd_kernel(ScanParams p) {
  constexpr int S = N / 4;
  constexpr bool FULL = M == kFull;
  constexpr int EL = Loader<E, N, kTile>::EL;
  const int tid = threadIdx.x, lane = tid & 63, c = (tid >> 6) * 16 + (lane & 15), q = lane >> 4;
  const int n = blockIdx.z, seg = blockIdx.y;
  const ChannelTile ct(p, blockIdx.x);
  int64_t bos, len;
  chunk::seq_range(p.seq, n, bos, len);
  const int last = len > 0 ? static_cast<int>((len - 1) / p.seg_len) : 0;
  if (FULL ? seg > last : seg >= last) return;
  const int64_t begin = seg * p.seg_len, end = min(len, begin + p.seg_len);

  __shared__ Stage<N, kTile> stage[2];
  __shared__ ChannelParams cp;
  __shared__ float ybuf[FULL ? 2 : 1][FULL ? kTile : 1][kYStride];
  __shared__ float sums[FULL ? 1 : 4][kScanTile];

  // this lane's states: channel ct.d0 + c, states q S .. q S + S - 1
  const bool chan = c < ct.count;
  const int64_t hd = static_cast<int64_t>(ct.d0 + c) * N + q * S;
  float A2[S], h[S];
  load_states<S>(p.A + hd, chan, A2);
#pragma unroll
  for (int s = 0; s < S; ++s) A2[s] *= kLog2e;
  if (FULL) {
    load_states<S>(p.h0 + static_cast<int64_t>(n) * p.D * N + hd, chan && p.h0, h);
    for (int g = 0; g < seg; ++g) {
      const int64_t part = part_slot(p, bos, n, g);
      const float sum = chan ? p.seg_sum[part * p.D + ct.d0 + c] : 0.f;
      float e[S];
      load_states<S>(p.seg_end + part * p.D * N + hd, chan, e);
#pragma unroll
      for (int s = 0; s < S; ++s) h[s] = fmaf(exp2_(A2[s] * sum), h[s], e[s]);
    }
  } else {
#pragma unroll
    for (int s = 0; s < S; ++s) h[s] = 0.f;
  }

  Loader<E, N, kTile> ld(p, ct, bos, FULL && p.z);
  float delta[EL], sig[EL];
  cp.fill(p, ct);
  __syncthreads();
  if (begin < end) {
    ld.fetch(begin, end);
    ld.put(stage[0], cp, begin, end, delta, sig);
  }
  float dsum = 0.f;  // kSummary: delta of this thread's channel over a quarter of the tokens
  __syncthreads();
  int b = 0;
  for (int64_t t0 = begin; t0 < end; t0 += kTile, b ^= 1) {
    const Raw<E, EL> ru = ld.u, rz = ld.z;
    const bool more = t0 + kTile < end;
    if (more) ld.fetch(t0 + kTile, end);
    const Stage<N, kTile>& st = stage[b];
#pragma unroll 2
    for (int t = 0; t < kTile; t += 4) {
      __builtin_amdgcn_s_setprio(2);
      if (FULL && t % kScanBlock == 0 && p.saved && t0 + t < end && chan)
        store_states<S>(p.saved + saved_slot(bos, n, t0 + t) * p.D * N + hd, h);
      // four tokens' decays and writes first, then the chain through them: a wave
      // has independent work while an exponential is on its way
      float a[4][S], w[4][S], acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 dd = st.dd[t + j][c];
        float Bv[S];
        read_states<S>(&st.B[t + j][q * S], Bv);
#pragma unroll
        for (int s = 0; s < S; ++s) {
          a[j][s] = dd.x * A2[s];
          w[j][s] = dd.y * Bv[s];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int s = 0; s < S; ++s) a[j][s] = exp2_(a[j][s]);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float Cv[S];
        if (FULL) read_states<S>(&st.C[t + j][q * S], Cv);
        acc[j] = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
          h[s] = fmaf(a[j][s], h[s], w[j][s]);
          if (FULL) acc[j] = fmaf(h[s], Cv[s], acc[j]);
        }
      }
      if (FULL) ybuf[b][t + q][c] = reduce_rows4(acc[0], acc[1], acc[2], acc[3]);
    }
    __builtin_amdgcn_s_setprio(0);
    if (!FULL) {
#pragma unroll
      for (int t = 0; t < kTile; t += 4) dsum += st.dd[t + q][c].x;
    }
    if (more) ld.put(stage[b ^ 1], cp, t0 + kTile, end, delta, sig);
    __syncthreads();
    if (FULL) {
      const int64_t t = t0 + ld.row;
      if (t < end && ld.live) {
        const float* const yr = &ybuf[b][ld.row][ld.col];
        float y[EL];
#pragma unroll
        for (int e = 0; e < EL; ++e) {
          y[e] = fmaf(cp.skip[ld.col + e], ru.get(e), yr[e]);
          if (p.z) {
            const float z = rz.get(e);
            y[e] *= z * sigmoid_(z);
          }
        }
        store_vec<E, EL>(static_cast<E*>(p.y) + (bos + t) * p.D + ct.d0 + ld.col, y);
      }
    }
  }
  if (FULL) {
    if (seg == last && p.h_final && chan) store_states<S>(p.h_final + static_cast<int64_t>(n) * p.D * N + hd, h);
  } else {
    const int64_t part = part_slot(p, bos, n, seg);
    if (chan) store_states<S>(p.seg_end + part * p.D * N + hd, h);
    sums[q][c] = dsum;
    __syncthreads();
    if (tid < kScanTile && tid < ct.count)
      p.seg_sum[part * p.D + ct.d0 + tid] = (sums[0][tid] + sums[1][tid]) + (sums[2][tid] + sums[3][tid]);
  }
}

// One token: four lanes a channel, N / 4 contiguous states each (a wave covers 16
// channels' states as one contiguous piece).  The state is read and written once: 64 x
// 4096 x 16, 36 MB, takes 9.1 us (4.0 TB/s); two, four or eight sequences a thread take
// as long or longer.
template <typename E, int N>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanParams p) {
  constexpr int S = N / 4;
  const int tid = threadIdx.x, q = tid & 3;
  const int d = blockIdx.x * 64 + (tid >> 2);
  if (d >= p.D) return;  // whole groups of four lanes
  const int64_t b = blockIdx.y, bd = b * p.D + d;
  const int64_t bc = (b * p.G + d / (p.D / p.G)) * N + q * S;
  float A[S], h[S], Bv[S], Cv[S];
  load_states<S>(p.h_final + bd * N + q * S, true, h);
  load_states<S>(p.A + static_cast<int64_t>(d) * N + q * S, true, A);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    Bv[s] = IoT<E>::ld(static_cast<const E*>(p.Bm) + bc + s);
    Cv[s] = IoT<E>::ld(static_cast<const E*>(p.Cm) + bc + s);
  }
  const float u = IoT<E>::ld(static_cast<const E*>(p.u) + bd);
  float delta = IoT<E>::ld(static_cast<const E*>(p.dt) + bd) + (p.dt_bias ? p.dt_bias[d] : 0.f);
  const float skip = p.Dskip ? p.Dskip[d] : 0.f;
  const float z = p.z ? IoT<E>::ld(static_cast<const E*>(p.z) + bd) : 0.f;
  float sig;
  if (p.softplus) delta = softplus_(delta, sig);
  const float du = delta * u;
  float y = 0.f;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    h[s] = fmaf(exp2_(delta * (A[s] * kLog2e)), h[s], du * Bv[s]);
    y = fmaf(h[s], Cv[s], y);
  }
  store_states<S>(p.h_final + bd * N + q * S, h);
  y += dpp_f32<0xB1, 0xf>(y);  // quad_perm 1,0,3,2
  y += dpp_f32<0x4E, 0xf>(y);  // quad_perm 2,3,0,1
  if (q == 0) {
    y = fmaf(skip, u, y);
    if (p.z) y *= z * sigmoid_(z);
    IoT<E>::st(static_cast<E*>(p.y) + bd, y);
  }
}

template <typename E, int N>
hipError_t fwd_t(const ScanParams& p, hipStream_t s) {
  const unsigned tiles = static_cast<unsigned>(scan_tiles(p.D, p.G)), nseq = static_cast<unsigned>(p.nseq);
  if (p.segs > 1)
    hipLaunchKernelGGL((scan_fwd_kernel<E, N, kSummary>), dim3(tiles, p.segs - 1, nseq), dim3(256), 0, s, p);
  hipLaunchKernelGGL((scan_fwd_kernel<E, N, kFull>), dim3(tiles, p.segs, nseq), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename E, int N>
hipError_t step_t(const ScanParams& p, hipStream_t s) {
  hipLaunchKernelGGL((scan_step_kernel<E, N>), dim3((p.D + 63) / 64, static_cast<unsigned>(p.nseq)), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_fwd(const ScanParams& p, int N, bool bf16, hipStream_t s) {
  if (p.in_time) return launch_scan_time(p, N, bf16, s);
  GDN_SCAN_DISPATCH(fwd_t)
}
hipError_t launch_scan_step(const ScanParams& p, int N, bool bf16, hipStream_t s) { GDN_SCAN_DISPATCH(step_t) }

}  // namespace gdn
