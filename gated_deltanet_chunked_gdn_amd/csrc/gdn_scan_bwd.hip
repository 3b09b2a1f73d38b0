// Backward of the selective scan on gfx950, from the states the forward kept every 16
// tokens.  With ds = dy silu(z) and G the gradient of the state after a token
// (G_t = C_t ds_t + a_{t+1} G_{t+1}, from dh_final behind the last token):
//     dC_t = sum_d h_t ds_t          dB_t = sum_d G_t delta u
//     du = D ds + delta sum_n G B    ddelta = u sum_n G B + sum_n A q,  q = G a h_{t-1}
//     dA = sum_t delta q             dz = dy s silu'(z),  s = sum_n C h + D u
//
// Blocks of 16 tokens go from the last to the first.  Of a block, every lane forms
// its states and decays forward from the kept state (they stay in registers: 16
// tokens x 4 states x 2) and then walks back; wider states take the block four states
// a lane at a time.  The work is bound by vector instructions, as the forward, with
// the sums over the channels on top: a lane's 16 values of dB (four tokens, four
// states) are added over the 16 channels of its wave by lane swaps that halve the
// registers each time (rows of 16 lanes hold channels c / 4: two swap steps), then by
// two DPP adds inside the quad that holds channels c % 4.  Each workgroup writes its
// 64 channels' sums of dB and dC, and one kernel adds them over the channel tiles in
// order; the sums of dA, dD and ddt_bias over the tokens are added over the segments
// and sequences by another.  No atomics: the same inputs give the same bits.
#include <hip/hip_runtime.h>

#include "gdn_scan_device.h"

namespace gdn {
namespace {

using namespace layer;
using namespace scan;

constexpr int TT = kScanBlock;

// Sum over the four lanes of a quad (channels c % 4), in all four.
__device__ __forceinline__ float quad_sum(float x) {
  x += dpp_f32<0xB1, 0xf>(x);  // quad_perm 1,0,3,2
  x += dpp_f32<0x4E, 0xf>(x);  // quad_perm 2,3,0,1
  return x;
}
// Sum over the lanes of a row that differ in bits 2 and 3 (a channel's four lanes).
__device__ __forceinline__ float states_sum(float x) {
  x += dpp_f32<0x128, 0xf>(x);  // row_ror:8
  x += dpp_f32<0x124, 0xf>(x);  // row_ror:4
  return x;
}
// v[i] summed over the wave's channels: afterwards r[i], i < 4, of a lane in row rr
// holds v[4 rr + i] (of the lane's states).
__device__ __forceinline__ void channels_sum16(float (&v)[16], float (&r)[4]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    swap32(v[i], v[i + 8]);
    v[i] += v[i + 8];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    swap16(v[i], v[i + 4]);
    r[i] = quad_sum(v[i] + v[i + 4]);
  }
}

// This lane's place: channel c of the tile's 64, quarter q of its states.
struct Place {
  int c, q;
  __device__ __forceinline__ Place() {
    const int lane = threadIdx.x & 63;
    c = (threadIdx.x >> 6) * 16 + (lane >> 4) * 4 + (lane & 3);
    q = (lane >> 2) & 3;
  }
};

// ds of a tile: dy, or dy silu(z).
template <typename E, int N>
struct BwdLoader : Loader<E, N, TT> {
  using L = Loader<E, N, TT>;
  static constexpr int EL = L::EL;
  Raw<E, EL> dy;
  __device__ __forceinline__ BwdLoader(const ScanParams& p, const ChannelTile& ct, int64_t bos)
      : L(p, ct, bos, p.z != nullptr) {}
  __device__ __forceinline__ void fetch(int64_t t0, int64_t end) {
    L::fetch(t0, end);
    dy.load(static_cast<const E*>(this->p.dy) + this->token(t0, end) * this->p.D + this->d);
  }
  __device__ __forceinline__ void put_ds(float (&ds)[TT][kScanTile], int64_t t0, int64_t end, float (&f)[EL]) const {
    const bool both = t0 + this->row < end && this->live;
#pragma unroll
    for (int e = 0; e < EL; ++e) {
      float g = dy.get(e);
      if (this->has_z) {
        const float z = this->z.get(e);
        g *= z * sigmoid_(z);
      }
      f[e] = both ? g : 0.f;
    }
    *reinterpret_cast<float4*>(&ds[this->row][this->col]) = float4{f[0], f[1], f[2], f[3]};
  }
};

// Gradient of the state before every segment but the first of a sequence, from a zero
// gradient behind it, and the segment's sum of delta.
template <typename E, int N>
__global__ __launch_bounds__(256) void scan_bwd_summary_kernel(ScanParams p) {
  constexpr int S = N / 4, EL = BwdLoader<E, N>::EL;
  const int tid = threadIdx.x;
  const Place at;
  const int n = blockIdx.z, seg = blockIdx.y + 1;
  const ChannelTile ct(p, blockIdx.x);
  int64_t bos, len;
  chunk::seq_range(p.seq, n, bos, len);
  const int64_t begin = seg * p.seg_len, end = min(len, begin + p.seg_len);
  if (begin >= end) return;

  __shared__ Stage<N, TT> st;
  __shared__ float dsb[TT][kScanTile];
  __shared__ float sums[4][kScanTile];
  const bool chan = at.c < ct.count;
  const int64_t hd = static_cast<int64_t>(ct.d0 + at.c) * N + at.q * S;
  float A2[S], G[S];
  load_states<S>(p.A + hd, chan, A2);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    A2[s] *= kLog2e;
    G[s] = 0.f;
  }
  float dsum = 0.f, delta[EL], sig[EL], ds[EL];
  BwdLoader<E, N> ld(p, ct, bos);
  int64_t t0 = begin + (end - begin - 1) / TT * TT;
  ld.fetch(t0, end);
  for (; t0 >= begin; t0 -= TT) {
    ld.put(st, t0, end, delta, sig);
    ld.put_ds(dsb, t0, end, ds);
    if (t0 > begin) ld.fetch(t0 - TT, end);
    __syncthreads();
#pragma unroll
    for (int t = TT - 1; t >= 0; --t) {
      const float d = st.dd[t][at.c].x, g = dsb[t][at.c];
      float Cv[S];
      read_states<S>(&st.C[t][at.q * S], Cv);
#pragma unroll
      for (int s = 0; s < S; ++s) G[s] = exp2_(d * A2[s]) * fmaf(Cv[s], g, G[s]);
      if (t % 4 == at.q) dsum += d;
    }
    __syncthreads();
  }
  const int64_t part = static_cast<int64_t>(seg) * p.nseq + n;
  if (chan) store_states<S>(p.seg_end + part * p.D * N + hd, G);
  sums[at.q][at.c] = dsum;
  __syncthreads();
  if (tid < kScanTile && tid < ct.count)
    p.seg_sum[part * p.D + ct.d0 + tid] = (sums[0][tid] + sums[1][tid]) + (sums[2][tid] + sums[3][tid]);
}

template <typename E, int N>
__global__ __launch_bounds__(256) void scan_bwd_kernel(ScanParams p) {
  constexpr int S = N / 4;
  constexpr int SG = S < 4 ? S : 4;  // states of a lane taken at a time
  constexpr int TG = 16 / SG;        // tokens whose dB, dC are summed together
  constexpr int EL = BwdLoader<E, N>::EL;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const Place at;
  const int n = blockIdx.z, seg = blockIdx.y;
  const ChannelTile ct(p, blockIdx.x);
  int64_t bos, len;
  chunk::seq_range(p.seq, n, bos, len);
  const int last = len > 0 ? static_cast<int>((len - 1) / p.seg_len) : 0;
  const int64_t begin = seg * p.seg_len, end = min(len, begin + p.seg_len);
  const int64_t part = static_cast<int64_t>(seg) * p.nseq + n;

  __shared__ Stage<N, TT> st;
  __shared__ float dsb[TT][kScanTile];
  __shared__ float gB[TT][kScanTile], Aq[TT][kScanTile], Ch[TT][kScanTile];  // sums over a channel's states
  __shared__ float bc[4][TT][2][N];                                         // dB, dC of each wave's channels

  const bool chan = at.c < ct.count;
  const int64_t hd = static_cast<int64_t>(ct.d0 + at.c) * N + at.q * S;
  float A2[S], G[S], dA[S];
  load_states<S>(p.A + hd, chan, A2);
  load_states<S>(p.dh_final + static_cast<int64_t>(n) * p.D * N + hd, chan && p.dh_final, G);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    A2[s] *= kLog2e;
    dA[s] = 0.f;
  }
  for (int g = last; g > seg; --g) {
    const int64_t pt = static_cast<int64_t>(g) * p.nseq + n;
    const float sum = chan ? p.seg_sum[pt * p.D + ct.d0 + at.c] : 0.f;
    float e[S];
    load_states<S>(p.seg_end + pt * p.D * N + hd, chan, e);
#pragma unroll
    for (int s = 0; s < S; ++s) G[s] = fmaf(exp2_(A2[s] * sum), G[s], e[s]);
  }

  float delta[EL], sig[EL], ds[EL], dD[EL], dbias[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) dD[e] = dbias[e] = 0.f;
  BwdLoader<E, N> ld(p, ct, bos);
  int64_t t0 = begin + (end - begin - 1) / TT * TT;
  if (begin < end) ld.fetch(t0, end);
  for (; begin < end && t0 >= begin; t0 -= TT) {
    float h0[S];
    load_states<S>(p.saved + saved_slot(bos, n, t0) * p.D * N + hd, chan, h0);
    ld.put(st, t0, end, delta, sig);
    ld.put_ds(dsb, t0, end, ds);
    const Raw<E, EL> ru = ld.u, rz = ld.z, rdy = ld.dy;
    if (t0 > begin) ld.fetch(t0 - TT, end);
    __syncthreads();
#pragma unroll
    for (int s0 = 0; s0 < S; s0 += SG) {
      float a[TT][SG], hb[TT + 1][SG];  // decay of a token, state before it
#pragma unroll
      for (int s = 0; s < SG; ++s) hb[0][s] = h0[s0 + s];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const float2 dd = st.dd[t][at.c];
        float Bv[SG];
        read_states<SG>(&st.B[t][at.q * S + s0], Bv);
#pragma unroll
        for (int s = 0; s < SG; ++s) {
          a[t][s] = exp2_(dd.x * A2[s0 + s]);
          hb[t + 1][s] = fmaf(a[t][s], hb[t][s], dd.y * Bv[s]);
        }
      }
#pragma unroll
      for (int tg = TT - TG; tg >= 0; tg -= TG) {
        float vB[16], vC[16];
#pragma unroll
        for (int tt = TG - 1; tt >= 0; --tt) {
          const int t = tg + tt;
          const float2 dd = st.dd[t][at.c];
          const float g = dsb[t][at.c];
          float Bv[SG], Cv[SG];
          read_states<SG>(&st.B[t][at.q * S + s0], Bv);
          read_states<SG>(&st.C[t][at.q * S + s0], Cv);
          float sB = 0.f, sA = 0.f, sC = 0.f;
#pragma unroll
          for (int s = 0; s < SG; ++s) {
            float& Gs = G[s0 + s];
            Gs = fmaf(Cv[s], g, Gs);
            vC[tt * SG + s] = hb[t + 1][s] * g;
            vB[tt * SG + s] = Gs * dd.y;
            sC = fmaf(hb[t + 1][s], Cv[s], sC);
            sB = fmaf(Gs, Bv[s], sB);
            Gs *= a[t][s];
            const float qv = Gs * hb[t][s];
            sA = fmaf(A2[s0 + s], qv, sA);
            dA[s0 + s] = fmaf(dd.x, qv, dA[s0 + s]);
          }
          sB = states_sum(sB);
          sA = states_sum(sA);
          sC = states_sum(sC);
          // the four lanes of a channel hold the same sums: each writes one (or none)
          float* const to = at.q == 0 ? &gB[t][at.c] : at.q == 1 ? &Aq[t][at.c] : &Ch[t][at.c];
          const float val = at.q == 0 ? sB : at.q == 1 ? sA : sC;
          if (at.q < 3) *to = s0 == 0 ? val : *to + val;
        }
        float rB[4], rC[4];
        channels_sum16(vB, rB);
        channels_sum16(vC, rC);
        if ((lane & 3) == 0) {
          // value 4 rr + i of a group is state i % SG of token tg + (4 rr + i) / SG
          const int rr = lane >> 4;
          if constexpr (SG == 4) {
            store_states<4>(&bc[wave][tg + rr][0][at.q * S + s0], rB);
            store_states<4>(&bc[wave][tg + rr][1][at.q * S + s0], rC);
          } else {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              *reinterpret_cast<float2*>(&bc[wave][tg + 2 * rr + i / 2][0][at.q * S]) = float2{rB[i], rB[i + 1]};
              *reinterpret_cast<float2*>(&bc[wave][tg + 2 * rr + i / 2][1][at.q * S]) = float2{rC[i], rC[i + 1]};
            }
          }
        }
      }
    }
    __syncthreads();
    const int64_t t = t0 + ld.row;
    if (t < end && ld.live) {
      const int64_t off = (bos + t) * p.D + ct.d0 + ld.col;
      float du[EL], ddt[EL], dz[EL];
#pragma unroll
      for (int e = 0; e < EL; ++e) {
        const float u = ru.get(e), sB = gB[ld.row][ld.col + e], sA = Aq[ld.row][ld.col + e] * (1.f / kLog2e);
        du[e] = fmaf(ld.skip[e], ds[e], delta[e] * sB);
        ddt[e] = fmaf(u, sB, sA) * sig[e];
        dD[e] = fmaf(ds[e], u, dD[e]);
        dbias[e] += ddt[e];
        if (ld.has_z) {
          const float z = rz.get(e), sg = sigmoid_(z);
          dz[e] = rdy.get(e) * fmaf(ld.skip[e], u, Ch[ld.row][ld.col + e]) * (sg * fmaf(z, 1.f - sg, 1.f));
        }
      }
      store_vec<E, EL>(static_cast<E*>(p.du) + off, du);
      store_vec<E, EL>(static_cast<E*>(p.ddt) + off, ddt);
      if (p.dz) store_vec<E, EL>(static_cast<E*>(p.dz) + off, dz);
    }
    for (int i = tid; i < TT * 2 * N; i += 256) {
      const int row = i / (2 * N), k = i % (2 * N);
      if (t0 + row < end) {
        const float* const w = &bc[0][row][0][0] + k;
        p.part_bc[((static_cast<int64_t>(ct.tile) * p.rows + bos + t0 + row) * p.G + ct.g) * 2 * N + k] =
            (w[0] + w[TT * 2 * N]) + (w[2 * TT * 2 * N] + w[3 * TT * 2 * N]);
      }
    }
  }
  // what goes over the tokens: dA of this lane's states, dD and ddt_bias of the tile's channels
  const int64_t pa = (part * p.D + ct.d0) * (N + 2);
  if (chan) {
#pragma unroll
    for (int s = 0; s < S; ++s) p.part_a[pa + at.c * (N + 2) + at.q * S + s] = dA[s];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < EL; ++e) {
    gB[ld.row][ld.col + e] = dD[e];
    Aq[ld.row][ld.col + e] = dbias[e];
  }
  __syncthreads();
  if (tid < 2 * kScanTile) {
    const int c = tid % kScanTile, k = tid / kScanTile;
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < TT; ++r) sum += k ? Aq[r][c] : gB[r][c];
    if (c < ct.count) p.part_a[pa + c * (N + 2) + N + k] = sum;
  }
  if (seg == 0 && p.dh0 && chan) store_states<S>(p.dh0 + static_cast<int64_t>(n) * p.D * N + hd, G);
}

// dB and dC: the channel tiles' sums in order.
template <typename E, int N>
__global__ __launch_bounds__(256) void scan_bwd_bc_kernel(ScanParams p, int tiles, int64_t items) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= items) return;
  float s = 0.f;
  for (int k = 0; k < tiles; ++k) s += p.part_bc[static_cast<int64_t>(k) * items + i];
  const int64_t rg = i / (2 * N);
  const int k = static_cast<int>(i % (2 * N));
  E* const out = static_cast<E*>(k < N ? p.dBm : p.dCm);
  IoT<E>::st(out + rg * N + k % N, s);
}

// dA, dDskip and ddt_bias: the segments' and sequences' sums in order.
template <int N>
__global__ __launch_bounds__(256) void scan_bwd_a_kernel(ScanParams p, int64_t parts) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, items = static_cast<int64_t>(p.D) * (N + 2);
  if (i >= items) return;
  float s = 0.f;
  for (int64_t k = 0; k < parts; ++k) s += p.part_a[k * items + i];
  const int64_t d = i / (N + 2);
  const int k = static_cast<int>(i % (N + 2));
  if (k < N)
    p.dA[d * N + k] = s;
  else if (k == N) {
    if (p.dDskip) p.dDskip[d] = s;
  } else if (p.ddt_bias) {
    p.ddt_bias[d] = s;
  }
}

unsigned blocks_of(int64_t threads) { return static_cast<unsigned>((threads + 255) / 256); }

template <typename E, int N>
hipError_t bwd_t(const ScanParams& p, hipStream_t s) {
  const unsigned tiles = static_cast<unsigned>(scan_tiles(p.D, p.G)), nseq = static_cast<unsigned>(p.nseq);
  if (nseq > 0) {
    if (p.segs > 1)
      hipLaunchKernelGGL((scan_bwd_summary_kernel<E, N>), dim3(tiles, p.segs - 1, nseq), dim3(256), 0, s, p);
    hipLaunchKernelGGL((scan_bwd_kernel<E, N>), dim3(tiles, p.segs, nseq), dim3(256), 0, s, p);
  }
  const int64_t items = p.rows * p.G * 2 * N;
  if (items > 0)
    hipLaunchKernelGGL((scan_bwd_bc_kernel<E, N>), dim3(blocks_of(items)), dim3(256), 0, s, p,
                       static_cast<int>(tiles / p.G), items);
  hipLaunchKernelGGL((scan_bwd_a_kernel<N>), dim3(blocks_of(static_cast<int64_t>(p.D) * (N + 2))), dim3(256), 0, s, p,
                     static_cast<int64_t>(p.segs) * p.nseq);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_bwd(const ScanParams& p, int N, bool bf16, hipStream_t s) {
  switch (N) {
    case 8: return bf16 ? bwd_t<uint16_t, 8>(p, s) : bwd_t<float, 8>(p, s);
    case 16: return bf16 ? bwd_t<uint16_t, 16>(p, s) : bwd_t<float, 16>(p, s);
    case 32: return bf16 ? bwd_t<uint16_t, 32>(p, s) : bwd_t<float, 32>(p, s);
    default: return bf16 ? bwd_t<uint16_t, 64>(p, s) : bwd_t<float, 64>(p, s);
  }
}

}  // namespace gdn
