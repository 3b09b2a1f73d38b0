// The selective scan's forward with the time axis inside the workgroup, on gfx950.
//
// Four waves hold the same 16 channels (8 of 32 states, 4 of 64: four states a lane) and
// take 16 consecutive tokens each, 64 a step.  A wave forms its tokens' decays a and
// writes w = delta u B once, keeps them in registers (16 tokens x 4 states x 2) while it runs h <- a h + w from zero to its
// end, and passes (product of the decays, end state) through LDS.  Every wave then folds
// the four pairs onto the carried state, which gives its own start and the next step's
// carry, and runs its tokens again from the start: two more multiply-adds a state (the
// second with C) instead of another pass with the exponentials.  So the time axis is
// parallel at six vector instructions per token, channel and state, where the split
// over segments (gdn_scan.hip) spends nine, and the staging twice.
//
// Measured, bf16, 16 states, forward: 2 x 2048 x 4096 90 us a call where calls queue up (100
// without the wave priorities), 98 to 109 us a launch by itself in a trace (9.6 vector instructions a token, channel and state with the staging and the
// gate, at the two waves a SIMD that the registers leave), 1 x 128 x 1024 7 us (10 us
// split: one launch instead of two).  64 states, six
// packed prompts, 3001 x 1024: 75 us (93 us split).  Eight waves of eight tokens, at four
// waves a SIMD, gain nothing (131 us for the first, the same for the last): they fold twice
// as often.
//
// Each wave stages its own tokens; one barrier a step, for the pairs.  Workgroups of
// neighbouring channels share cache lines (row pieces of 8 to 64 bytes), so each XCD takes
// an eighth of the channels: its workgroups follow each other eight apart in the grid.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "gdn_scan_device.h"

namespace gdn {
namespace {

using namespace layer;
using namespace scan;

constexpr int kTok = 16;   // tokens of a wave
constexpr int kStep = 64;  // tokens of a step

// One or two values as loaded (Raw takes whole vectors of 8 or 16 bytes).
template <typename E, int NV>
struct alignas(NV * sizeof(E)) Few {
  E v[NV];
  __device__ __forceinline__ void load(const E* p) { *this = *reinterpret_cast<const Few*>(p); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = E(0);
  }
  __device__ __forceinline__ float get(int e) const { return IoT<E>::ld(&v[e]); }
};
template <typename E, int NV>
using Vals = std::conditional_t<NV * sizeof(E) >= 8, Raw<E, NV>, Few<E, NV>>;

template <typename E, int N>
__global__ __launch_bounds__(256, 2) void scan_time_kernel(ScanParams p, int tiles) {
  constexpr int kCh = scan_time_channels(N), EL = kCh / 4;
  constexpr int S = kCh * N / 64, P = N / 4;  // states of a lane; a lane's values of one token's B and C
  // stride of B and C rows: the rows that a wave writes at once fall in other banks
  constexpr int kRow = N > 16 ? N + 4 : N;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane % kCh, q = lane / kCh;
  const int n = blockIdx.y;
  // tile: 8 XCDs take workgroups in turn, so workgroups x, x + 8, ... share one
  const int x = blockIdx.x, per = (tiles + 7) / 8, tile = (x & 7) * per + (x >> 3);
  if (tile >= tiles) return;
  const int dg = p.D / p.G, tg = (dg + kCh - 1) / kCh, g = tile / tg;
  const int at = (tile - g * tg) * kCh, d0 = g * dg + at, count = min(kCh, dg - at);
  int64_t bos, len;
  chunk::seq_range(p.seq, n, bos, len);

  __shared__ alignas(16) float2 dd[4][kTok][kCh];
  __shared__ alignas(16) float Bs[4][kTok][kRow], Cs[4][kTok][kRow];
  __shared__ alignas(16) float ys[4][kTok][kCh + 4];
  __shared__ float pair[2][4][2][64][S];  // decay product, end state of each wave

  const bool chan = c < count;
  const int64_t hd = static_cast<int64_t>(d0 + c) * N + q * S;
  float A2[S], carry[S];
  load_states<S>(p.A + hd, chan, A2);
  load_states<S>(p.h0 + static_cast<int64_t>(n) * p.D * N + hd, chan && p.h0, carry);
#pragma unroll
  for (int s = 0; s < S; ++s) A2[s] *= kLog2e;

  // this lane's share of the wave's tile: a quarter of the channels of one token
  const int row = lane >> 2, piece = lane & 3, col = piece * EL;
  const bool live = col < count;
  const int d = d0 + (live ? col : 0);
  Vals<float, EL> bias, skip;
  bias.zero();
  skip.zero();
  if (p.dt_bias) bias.load(p.dt_bias + d);
  if (p.Dskip) skip.load(p.Dskip + d);
  Vals<E, EL> ru, rdt, rz;
  Vals<E, P> rb, rc;
  auto fetch = [&](int64_t t0) {
    const int64_t t = bos + min(t0 + wave * kTok + row, len - 1);
    ru.load(static_cast<const E*>(p.u) + t * p.D + d);
    rdt.load(static_cast<const E*>(p.dt) + t * p.D + d);
    if (p.z) rz.load(static_cast<const E*>(p.z) + t * p.D + d);
    const int64_t bc = (t * p.G + g) * N + piece * P;
    rb.load(static_cast<const E*>(p.Bm) + bc);
    rc.load(static_cast<const E*>(p.Cm) + bc);
  };
  if (len > 0) fetch(0);
  int buf = 0;
  for (int64_t t0 = 0; t0 < len; t0 += kStep, buf ^= 1) {
    const int64_t t = t0 + wave * kTok + row;
    const bool ok = t < len;
    const Vals<E, EL> cu = ru, cz = rz;
    float delta[EL], sig;
#pragma unroll
    for (int e = 0; e < EL; ++e) delta[e] = rdt.get(e) + bias.get(e);
    if (p.softplus) {
#pragma unroll
      for (int e = 0; e < EL; ++e) delta[e] = softplus_(delta[e], sig);
    }
    if constexpr (EL == 1) {
      dd[wave][row][col] = ok && live ? float2{delta[0], delta[0] * cu.get(0)} : float2{0.f, 0.f};
    } else {
#pragma unroll
      for (int e = 0; e < EL; e += 2) {
        float4 v = {delta[e], delta[e] * cu.get(e), delta[e + 1], delta[e + 1] * cu.get(e + 1)};
        if (!ok || !live) v = float4{0.f, 0.f, 0.f, 0.f};
        *reinterpret_cast<float4*>(&dd[wave][row][col + e]) = v;
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      Bs[wave][row][piece * P + i] = ok ? rb.get(i) : 0.f;
      Cs[wave][row][piece * P + i] = ok ? rc.get(i) : 0.f;
    }
    if (t0 + kStep < len) fetch(t0 + kStep);
    __builtin_amdgcn_wave_barrier();

    // decays and writes, and the run from zero
    __builtin_amdgcn_s_setprio(1);
    float a[kTok][S], w[kTok][S], h[S], sum = 0.f;
#pragma unroll
    for (int s = 0; s < S; ++s) h[s] = 0.f;
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      const float2 v = dd[wave][j][c];
      float Bv[S];
      read_states<S>(&Bs[wave][j][q * S], Bv);
      sum += v.x;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        a[j][s] = exp2_(v.x * A2[s]);
        w[j][s] = v.y * Bv[s];
        h[s] = fmaf(a[j][s], h[s], w[j][s]);
      }
    }
    float prod[S];
#pragma unroll
    for (int s = 0; s < S; ++s) prod[s] = exp2_(A2[s] * sum);
    store_states<S>(pair[buf][wave][0][lane], prod);
    store_states<S>(pair[buf][wave][1][lane], h);
    __builtin_amdgcn_s_setprio(0);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k == wave) {
#pragma unroll
        for (int s = 0; s < S; ++s) h[s] = carry[s];
      }
      float e[S];
      read_states<S>(pair[buf][k][0][lane], prod);
      read_states<S>(pair[buf][k][1][lane], e);
#pragma unroll
      for (int s = 0; s < S; ++s) carry[s] = fmaf(prod[s], carry[s], e[s]);
    }
    const int64_t tw = t0 + wave * kTok;
    if (p.saved && tw < len && chan) store_states<S>(p.saved + saved_slot(bos, n, tw) * p.D * N + hd, h);
    // the run from its start, with the outputs
#pragma unroll
    for (int j = 0; j < kTok; j += 4) {
      float acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float Cv[S];
        read_states<S>(&Cs[wave][j + i][q * S], Cv);
        acc[i] = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
          h[s] = fmaf(a[j + i][s], h[s], w[j + i][s]);
          acc[i] = fmaf(h[s], Cv[s], acc[i]);
        }
      }
      // lanes of row t: token j + t; rotations by 8 and 4 lanes add the quarters of a row
      float yj = reduce_rows4(acc[0], acc[1], acc[2], acc[3]);
      if (kCh < 16) yj += dpp_f32<0x128, 0xf>(yj);
      if (kCh < 8) yj += dpp_f32<0x124, 0xf>(yj);
      if ((lane & 15) < kCh) ys[wave][j + (lane >> 4)][c] = yj;
    }
    __builtin_amdgcn_wave_barrier();
    if (ok && live) {
      Vals<float, EL> yv;
      yv.load(&ys[wave][row][col]);
      float y[EL];
#pragma unroll
      for (int e = 0; e < EL; ++e) {
        y[e] = fmaf(skip.get(e), cu.get(e), yv.get(e));
        if (p.z) {
          const float z = cz.get(e);
          y[e] *= z * sigmoid_(z);
        }
      }
      E* const to = static_cast<E*>(p.y) + (bos + t) * p.D + d;
      if constexpr (EL == 4) {
        store_vec<E, EL>(to, y);
      } else {
        Few<E, EL> out;
#pragma unroll
        for (int e = 0; e < EL; ++e) IoT<E>::st(&out.v[e], y[e]);
        *reinterpret_cast<Few<E, EL>*>(to) = out;
      }
    }
  }
  if (wave == 0 && p.h_final && chan) store_states<S>(p.h_final + static_cast<int64_t>(n) * p.D * N + hd, carry);
}

template <typename E, int N>
hipError_t launch_t(const ScanParams& p, hipStream_t s) {
  const int tiles = scan_time_tiles(p.D, p.G, N);
  hipLaunchKernelGGL((scan_time_kernel<E, N>), dim3((tiles + 7) / 8 * 8, static_cast<unsigned>(p.nseq)), dim3(256), 0, s,
                     p, tiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_time(const ScanParams& p, int N, bool bf16, hipStream_t s) {
  GDN_SCAN_DISPATCH(launch_t)
}

}  // namespace gdn
