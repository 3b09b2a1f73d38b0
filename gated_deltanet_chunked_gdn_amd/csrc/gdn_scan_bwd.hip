// Backward of the selective scan on gfx950, from the states the forward kept every 16
// tokens.  With ds = dy silu(z) and G the gradient of the state after a token
// (G_t = C_t ds_t + a_{t+1} G_{t+1}, from dh_final behind the last token):
//     dC_t = sum_d h_t ds_t          dB_t = sum_d G_t delta u
//     du = D ds + delta sum_n G B    ddelta = u sum_n G B + sum_n A q,  q = G a h_{t-1}
//     dA = sum_t delta q             dz = dy s silu'(z),  s = sum_n C h + D u
//
// Blocks of 16 tokens go from the last to the first.  Of a block, every lane forms its
// states and decays forward from the kept state (they stay in registers: 16 tokens x 4
// states x 2) and then walks back; wider states take the block four states a lane at a
// time, and G and dA wait in LDS between their passes.  All 256 registers of two waves a SIMD
// are taken from 16 states on, and what is held for a block's end goes to scratch in part:
// of the instances that form dz 0 (bf16) and 6 (fp32) registers with 16 states, 7 and 22 with
// 32, 7 and 34 with 64; of the others 1 and 9 with 16 and 64 fp32 states (up to four more in the
// instances for blocks that are not full).  The four lanes of a quad share a
// channel, so its sums over the states are two DPP exchanges; a lane's 16 values of dB
// (four tokens, four states) are added over the wave's 16 channels by steps that halve
// the values each time: two lane swaps over the rows of lanes, two exchanges between the
// quads of a row.  Each workgroup writes its 64 channels' sums of dB and dC, and a last
// kernel adds them over the channel tiles in order, and the sums of dA, dD and ddt_bias
// over the segments and sequences.  No atomics: the same inputs give the same bits.
//
// Bound by vector instructions, as the forward, with the sums over the channels on top:
// 22.7 a token, channel and state.  4 x 2048 tokens, 2048 channels, 16 states, bf16, with
// z: main kernel 201 to 204 us (222 without the wave priorities; the 345 MB it moves would
// take 67), summary of the segments 60, last kernel 11.  Measured
// and not kept: those sums by fp32 matrix instructions (381 us: the operands' layout
// costs more moves than the adds it saves), the rows of lanes added in LDS instead of by
// lane swaps (205 against 201), decays formed twice instead of kept, at three waves a SIMD
// (252).
#include <hip/hip_runtime.h>

#include "gdn_scan_device.h"

namespace gdn {
namespace {

using namespace layer;
using namespace scan;

constexpr int TT = kScanBlock;
// v[i], i < 16, summed over the wave's 16 channels: lane (cg, c3, q) gets value 4 cg + c3
// of its quarter q of the states.  Two lane swaps halve the registers while they add the
// rows of lanes (cg = c / 4), exchanges between the quads halve them over c % 4 = c3.
__device__ __forceinline__ float channels_sum16(float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    swap32(v[i], v[i + 8]);
    v[i] += v[i + 8];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    swap16(v[i], v[i + 4]);
    v[i] += v[i + 4];
  }
  // adds that write two of the four quads of a row each: quads 0, 1 keep v[0] and v[1] with
  // those of the quad two on, quads 2, 3 v[2] and v[3]; then the same between neighbours.
  // (A DPP operand may be read two wait states after it was written.)
  float x, y, sum;
  asm("s_nop 1\n\t"
      "v_add_f32_dpp %0, %3, %3 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %1, %4, %4 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %0, %5, %5 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %1, %6, %6 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "s_nop 1\n\t"
      "v_add_f32_dpp %2, %0, %0 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %2, %1, %1 row_shr:4 row_mask:0xf bank_mask:0xa"
      : "=&v"(x), "=&v"(y), "=&v"(sum)
      : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]));
  return sum;
}
// x[i], i < 4, summed over the four lanes of a channel (a quad): lane q gets x[q].
__device__ __forceinline__ float states_sum4(const float (&x)[4], bool q_hi, bool q_lo) {
  const float a = (q_hi ? x[2] : x[0]) + dpp_f32<0x4E, 0xf>(q_hi ? x[0] : x[2]);
  const float b = (q_hi ? x[3] : x[1]) + dpp_f32<0x4E, 0xf>(q_hi ? x[1] : x[3]);
  return (q_lo ? b : a) + dpp_f32<0xB1, 0xf>(q_lo ? a : b);
}

// The first pass over a block's states sets a sum, the others add to it.
template <int NG>
__device__ __forceinline__ void add_sum(float* to, float x, int pass) {
  *to = NG > 1 && pass > 0 ? *to + x : x;
}

// This lane's place: channel c of the tile's 64, quarter q of its states (the lanes of a
// quad share a channel, the four quads of a row hold channels c % 4).
struct Place {
  int c, q;
  __device__ __forceinline__ Place() {
    const int lane = threadIdx.x & 63;
    c = (threadIdx.x >> 6) * 16 + (lane >> 2);
    q = lane & 3;
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
// gradient behind it, and the segment's sum of delta.  Staged per (token, channel): delta
// and ds; two buffers, one barrier a block of 16 tokens.
template <typename E, int N>
__global__ __launch_bounds__(256) void scan_bwd_summary_kernel(ScanParams p) {
  constexpr int S = N / 4, EL = TT / 4, PC = N > 16 ? N / 16 : 1;
  const int tid = threadIdx.x;
  const Place at;
  const int n = blockIdx.z, seg = blockIdx.y + 1;
  const ChannelTile ct(p, blockIdx.x);
  int64_t bos, len;
  chunk::seq_range(p.seq, n, bos, len);
  const int64_t begin = seg * p.seg_len, end = min(len, begin + p.seg_len);
  if (begin >= end) return;

  __shared__ float2 dg[2][TT][kScanTile];
  __shared__ float Cs[2][TT][N];
  __shared__ float part[4][kScanTile];
  const bool chan = at.c < ct.count;
  const int64_t hd = static_cast<int64_t>(ct.d0 + at.c) * N + at.q * S;
  float A2[S], G[S];
  load_states<S>(p.A + hd, chan, A2);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    A2[s] *= kLog2e;
    G[s] = 0.f;
  }
  // a thread's share: four channels of one token, and a piece of its C
  const int row = tid >> 4, piece = tid & 15, col = piece * EL;
  const bool live = col < ct.count;
  const int d = ct.d0 + (live ? col : 0);
  Raw<float, EL> bias;
  bias.zero();
  if (p.dt_bias) bias.load(p.dt_bias + d);
  Raw<E, EL> rdt, rdy, rz;
  E rc[PC];
  auto fetch = [&](int64_t t0) {
    const int64_t t = bos + min(t0 + row, end - 1);
    rdt.load(static_cast<const E*>(p.dt) + t * p.D + d);
    rdy.load(static_cast<const E*>(p.dy) + t * p.D + d);
    if (p.z) rz.load(static_cast<const E*>(p.z) + t * p.D + d);
    const int64_t bc = (t * p.G + ct.g) * N + (piece * PC < N ? piece * PC : 0);
#pragma unroll
    for (int i = 0; i < PC; ++i) rc[i] = static_cast<const E*>(p.Cm)[bc + i];
  };
  auto put = [&](int b, int64_t t0) {
    const bool ok = t0 + row < end;
    float delta[EL], ds[EL], sig;
#pragma unroll
    for (int e = 0; e < EL; ++e) {
      delta[e] = rdt.get(e) + bias.get(e);
      ds[e] = rdy.get(e);
    }
    if (p.softplus) {
#pragma unroll
      for (int e = 0; e < EL; ++e) delta[e] = softplus_(delta[e], sig);
    }
    if (p.z) {
#pragma unroll
      for (int e = 0; e < EL; ++e) {
        const float z = rz.get(e);
        ds[e] *= z * sigmoid_(z);
      }
    }
#pragma unroll
    for (int e = 0; e < EL; e += 2) {
      float4 v = {delta[e], ds[e], delta[e + 1], ds[e + 1]};
      if (!ok || !live) v = float4{0.f, 0.f, 0.f, 0.f};
      *reinterpret_cast<float4*>(&dg[b][row][col + e]) = v;
    }
    if (piece * PC < N) {
#pragma unroll
      for (int i = 0; i < PC; ++i) Cs[b][row][piece * PC + i] = ok ? IoT<E>::ld(&rc[i]) : 0.f;
    }
  };
  int64_t t0 = begin + (end - begin - 1) / TT * TT;
  fetch(t0);
  put(0, t0);
  __syncthreads();
  float dsum = 0.f;
  for (int b = 0; t0 >= begin; t0 -= TT, b ^= 1) {
    if (t0 > begin) fetch(t0 - TT);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll 2
    for (int t = TT - 4; t >= 0; t -= 4) {
      // four tokens' decays first, then the chain through them
      float a[4][S], g[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = dg[b][t + j][at.c];
        g[j] = v.y;
        if (j == at.q) dsum += v.x;
#pragma unroll
        for (int s = 0; s < S; ++s) a[j][s] = exp2_(v.x * A2[s]);
      }
#pragma unroll
      for (int j = 3; j >= 0; --j) {
        float Cv[S];
        read_states<S>(&Cs[b][t + j][at.q * S], Cv);
#pragma unroll
        for (int s = 0; s < S; ++s) G[s] = a[j][s] * fmaf(Cv[s], g[j], G[s]);
      }
    }
    __builtin_amdgcn_s_setprio(0);
    if (t0 > begin) put(b ^ 1, t0 - TT);
    __syncthreads();
  }
  const int64_t pt = part_slot(p, bos, n, seg);
  if (chan) store_states<S>(p.seg_end + pt * p.D * N + hd, G);
  part[at.q][at.c] = dsum;
  __syncthreads();
  if (tid < kScanTile && tid < ct.count)
    p.seg_sum[pt * p.D + ct.d0 + tid] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
}

// G through the segments at `slot`, slot - 1, ... (`count` of them): sum and end are this
// lane's places in a slot of seg_sum and seg_end, its states NG pieces NW apart.  The
// loads of several segments are in flight together.
template <int NG, int SG>
__device__ __forceinline__ void compose(const ScanParams& p, const float* sum, const float* end, int64_t slot,
                                        int count, const float (&A2)[NG][SG], float (&G)[NG][SG]) {
  constexpr int M = NG * SG > 8 ? 2 : 4, NW = 4 * SG;
  const int64_t state = static_cast<int64_t>(p.D) * NG * NW;
  for (int i = 0; i < count; i += M) {
    float x[M], e[M][NG][SG];
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int64_t at = slot - min(i + j, count - 1);
      x[j] = sum[at * p.D];
#pragma unroll
      for (int k = 0; k < NG; ++k) load_states<SG>(end + at * state + k * NW, true, e[j][k]);
    }
#pragma unroll
    for (int j = 0; j < M; ++j) {
      if (i + j >= count) break;
#pragma unroll
      for (int k = 0; k < NG; ++k)
#pragma unroll
        for (int s = 0; s < SG; ++s) G[k][s] = fmaf(exp2_(A2[k][s] * x[j]), G[k][s], e[j][k][s]);
    }
  }
}

// GATED: dz is wanted, and with it the outputs before the gate.
// TAIL: a sequence's last block may have fewer than 16 tokens.  Tokens behind the end leave the
// state and G as they are and add delta G a h = 0 to dA, which a last state that is not finite
// would make NaN of: their states are set to zero.  Training steps without / with: 4 x 1999 x 1024
// channels, 32 states, bf16, 360 / 362 us; 4 x 1023 x 1000, 64 states, fp32, 369 / 383 us; four
// packed sequences, 777 x 320, 32 states, fp32, 52.9 / 54.0 us.
template <typename E, int N, bool GATED, bool TAIL>
__global__ __launch_bounds__(256, 2) void scan_bwd_kernel(ScanParams p) {
  constexpr int S = N / 4;
  constexpr int SG = S < 4 ? S : 4;  // states of a lane taken at a time
  constexpr int NG = S / SG;         // passes over a block
  constexpr int TG = 16 / SG;        // tokens whose dB, dC are summed together
  constexpr int NW = 4 * SG;         // states of a pass
  constexpr int EL = BwdLoader<E, N>::EL;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const Place at;
  const int n = blockIdx.z, seg = blockIdx.y;
  const ChannelTile ct(p, blockIdx.x);
  int64_t bos, len;
  chunk::seq_range(p.seq, n, bos, len);
  const int last = len > 0 ? static_cast<int>((len - 1) / p.seg_len) : 0;
  const int64_t begin = seg * p.seg_len, end = min(len, begin + p.seg_len);
  if (seg > last) return;
  const int64_t part = part_slot(p, bos, n, seg);

  __shared__ Stage<N, TT, 4> st;
  __shared__ ChannelParams cp;
  __shared__ float dsb[TT][kScanTile];
  __shared__ float sums[3][TT][kScanTile];   // over a channel's states: G B, A q, C h
  __shared__ float bc[4][TT][2][NW];         // dB, dC of each wave's channels, a pass
  __shared__ f32x4_t carry[NG > 1 ? 2 * NG : 1][NG > 1 ? 256 : 1];  // G and dA between a lane's passes

  const bool q_lo = lane & 1, q_hi = lane & 2;
  const int v16 = lane >> 2;  // the value of a group of 16 this lane gets
  const bool chan = at.c < ct.count;
  // the lane's states of pass k: q SG + NW k .. + SG - 1
  const int64_t hd = static_cast<int64_t>(ct.d0 + at.c) * N + at.q * SG;
  float A2[SG], G[SG], dA[SG];
  {
    float Ak[NG][SG], Gk[NG][SG];
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      load_states<SG>(p.A + hd + k * NW, chan, Ak[k]);
      load_states<SG>(p.dh_final + static_cast<int64_t>(n) * p.D * N + hd + k * NW, chan && p.dh_final, Gk[k]);
#pragma unroll
      for (int s = 0; s < SG; ++s) Ak[k][s] *= kLog2e;
    }
    if (chan)
      compose<NG, SG>(p, p.seg_sum + ct.d0 + at.c, p.seg_end + hd, part_slot(p, bos, n, last), last - seg, Ak, Gk);
#pragma unroll
    for (int s = 0; s < SG; ++s) {
      A2[s] = Ak[0][s];
      G[s] = Gk[0][s];
      dA[s] = 0.f;
    }
    if constexpr (NG > 1) {
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        carry[2 * k][tid] = f32x4_t{Gk[k][0], Gk[k][1], Gk[k][2], Gk[k][3]};
        carry[2 * k + 1][tid] = zero4();
      }
    }
  }

  float delta[EL], sig[EL], ds[EL], dD[EL], dbias[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) dD[e] = dbias[e] = 0.f;
  float* const part_bc = p.part_bc + ((static_cast<int64_t>(ct.tile) * p.rows + bos) * p.G + ct.g) * 2 * N;
  BwdLoader<E, N> ld(p, ct, bos);
  int64_t t0 = begin + (end - begin - 1) / TT * TT;
  float hn[SG];  // the kept state of the next pass
  const float* kept = p.saved + saved_slot(bos, n, t0) * p.D * N + hd;
  if (begin < end) {
    ld.fetch(t0, end);
    load_states<SG>(kept, chan, hn);
  }
  cp.fill(p, ct);
  // Lanes behind the tile's channels read B and C from four zeros behind each row: with the
  // real ones an infinity would make NaN of their zeros and reach the sums over the channels.
  if (tid < 4 * TT) {
    st.B[tid / 4][N + tid % 4] = 0.f;
    st.C[tid / 4][N + tid % 4] = 0.f;
  }
  __syncthreads();
  for (; begin < end && t0 >= begin; t0 -= TT) {
    ld.put(st, cp, t0, end, delta, sig);
    ld.put_ds(dsb, t0, end, ds);
    const Raw<E, EL> ru = ld.u, rz = ld.z, rdy = ld.dy;
    if (t0 > begin) ld.fetch(t0 - TT, end);
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < NG; ++k) {
      float a[TT][SG], hb[TT + 1][SG];  // a token's decay, the state before it
#pragma unroll
      for (int s = 0; s < SG; ++s) hb[0][s] = hn[s];
      if (k + 1 < NG) {
        load_states<SG>(kept + (k + 1) * NW, chan, hn);
      } else if (t0 > begin) {
        kept -= static_cast<int64_t>(p.D) * N;
        load_states<SG>(kept, chan, hn);
      }
      if constexpr (NG > 1) {
        const f32x4_t g4 = carry[2 * k][tid], a4 = carry[2 * k + 1][tid];
        load_states<SG>(p.A + hd + k * NW, chan, A2);
#pragma unroll
        for (int s = 0; s < SG; ++s) {
          G[s] = g4[s];
          dA[s] = a4[s];
          A2[s] *= kLog2e;
        }
      }
      // indexes the compiler cannot see through: on the way back the staged values are
      // read again rather than kept in (96) registers
      int ci = at.c, qi = chan ? at.q * SG + k * NW : N;
      __builtin_amdgcn_s_setprio(2);
#pragma unroll
      for (int tg = 0; tg < TT; tg += TG) {
        float v[16];
#pragma unroll
        for (int t4 = 0; t4 < TG; t4 += 4) {
          float sC[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int t = tg + t4 + j;
            const float2 dd = st.dd[t][ci];
            const float g = dsb[t][ci];
            float Bv[SG], Cv[SG];
            read_states<SG>(&st.B[t][qi], Bv);
            if (GATED) read_states<SG>(&st.C[t][qi], Cv);
            sC[j] = 0.f;
#pragma unroll
            for (int s = 0; s < SG; ++s) {
              a[t][s] = exp2_(dd.x * A2[s]);
              hb[t + 1][s] = fmaf(a[t][s], hb[t][s], dd.y * Bv[s]);
              v[(t4 + j) * SG + s] = hb[t + 1][s] * g;
              if (GATED) sC[j] = fmaf(hb[t + 1][s], Cv[s], sC[j]);
            }
          }
          if (GATED) add_sum<NG>(&sums[2][tg + t4 + at.q][at.c], states_sum4(sC, q_hi, q_lo), k);
        }
        bc[wave][tg + v16 / SG][1][at.q * SG + v16 % SG] = channels_sum16(v);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (TAIL && t0 + TT > end) {
#pragma unroll
        for (int t = 1; t < TT; ++t)
#pragma unroll
          for (int s = 0; s < SG; ++s) hb[t][s] = t0 + t < end ? hb[t][s] : 0.f;
      }
      asm volatile("" : "+v"(ci), "+v"(qi));
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int tg = TT - TG; tg >= 0; tg -= TG) {
        float v[16];
#pragma unroll
        for (int t4 = TG - 4; t4 >= 0; t4 -= 4) {
          float sB[4], sA[4];
#pragma unroll
          for (int j = 3; j >= 0; --j) {
            const int t = tg + t4 + j;
            const float2 dd = st.dd[t][ci];
            const float g = dsb[t][ci];
            float Bv[SG], Cv[SG];
            read_states<SG>(&st.B[t][qi], Bv);
            read_states<SG>(&st.C[t][qi], Cv);
            sB[j] = sA[j] = 0.f;
#pragma unroll
            for (int s = 0; s < SG; ++s) {
              G[s] = fmaf(Cv[s], g, G[s]);
              v[(t4 + j) * SG + s] = G[s] * dd.y;
              sB[j] = fmaf(G[s], Bv[s], sB[j]);
              G[s] *= a[t][s];
              const float qv = G[s] * hb[t][s];
              sA[j] = fmaf(A2[s], qv, sA[j]);
              dA[s] = fmaf(dd.x, qv, dA[s]);
            }
          }
          add_sum<NG>(&sums[0][tg + t4 + at.q][at.c], states_sum4(sB, q_hi, q_lo), k);
          add_sum<NG>(&sums[1][tg + t4 + at.q][at.c], states_sum4(sA, q_hi, q_lo), k);
        }
        bc[wave][tg + v16 / SG][0][at.q * SG + v16 % SG] = channels_sum16(v);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
      if constexpr (NG > 1) {
        carry[2 * k][tid] = f32x4_t{G[0], G[1], G[2], G[3]};
        carry[2 * k + 1][tid] = f32x4_t{dA[0], dA[1], dA[2], dA[3]};
      }
      __syncthreads();
      // the waves' sums
      if (tid < TT * 2 * NW / 4) {
        constexpr int kRow4 = 2 * NW / 4, kWave4 = TT * kRow4;
        const int row = tid / kRow4, x = tid % kRow4;
        const f32x4_t* const w = reinterpret_cast<const f32x4_t*>(&bc[0][0][0][0]) + tid;
        if (t0 + row < end)
          *reinterpret_cast<f32x4_t*>(part_bc + (t0 + row) * p.G * 2 * N + (x >= NW / 4 ? N : 0) + k * NW + x % (NW / 4) * 4) =
              (w[0] + w[kWave4]) + (w[2 * kWave4] + w[3 * kWave4]);
      }
      if (k + 1 < NG) __syncthreads();
    }
    const int64_t t = t0 + ld.row;
    if (t < end && ld.live) {
      const int64_t off = (bos + t) * p.D + ct.d0 + ld.col;
      float du[EL], ddt[EL], dz[EL];
#pragma unroll
      for (int e = 0; e < EL; ++e) {
        const float u = ru.get(e), sB = sums[0][ld.row][ld.col + e], sA = sums[1][ld.row][ld.col + e] * (1.f / kLog2e);
        du[e] = fmaf(cp.skip[ld.col + e], ds[e], delta[e] * sB);
        ddt[e] = fmaf(u, sB, sA) * sig[e];
        dD[e] = fmaf(ds[e], u, dD[e]);
        dbias[e] += ddt[e];
        if (GATED) {
          const float z = rz.get(e), sg = sigmoid_(z);
          dz[e] = rdy.get(e) * fmaf(cp.skip[ld.col + e], u, sums[2][ld.row][ld.col + e]) * (sg * fmaf(z, 1.f - sg, 1.f));
        }
      }
      store_vec<E, EL>(static_cast<E*>(p.du) + off, du);
      store_vec<E, EL>(static_cast<E*>(p.ddt) + off, ddt);
      if (GATED) store_vec<E, EL>(static_cast<E*>(p.dz) + off, dz);
    }
  }
  // what goes over the tokens: dA of this lane's states, dD and ddt_bias of the tile's channels
  float* const sums_a = p.part_a + (part * p.D + ct.d0) * (N + 2);
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    if constexpr (NG > 1) {
      const f32x4_t g4 = carry[2 * k][tid], a4 = carry[2 * k + 1][tid];
#pragma unroll
      for (int s = 0; s < SG; ++s) {
        G[s] = g4[s];
        dA[s] = a4[s];
      }
    }
    if (chan) {
#pragma unroll
      for (int s = 0; s < SG; ++s) sums_a[at.c * (N + 2) + k * NW + at.q * SG + s] = dA[s];
      if (seg == 0 && p.dh0) store_states<SG>(p.dh0 + static_cast<int64_t>(n) * p.D * N + hd + k * NW, G);
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < EL; ++e) {
    sums[0][ld.row][ld.col + e] = dD[e];
    sums[1][ld.row][ld.col + e] = dbias[e];
  }
  __syncthreads();
  if (tid < 2 * kScanTile) {
    const int c = tid % kScanTile, k = tid / kScanTile;
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < TT; ++r) sum += sums[k][r][c];
    if (c < ct.count) sums_a[c * (N + 2) + N + k] = sum;
  }
  if (seg == last) {  // slots that no segment has, up to the next sequence's
    const int64_t next = (bos + len) / p.seg_len + n + 1;
    for (int64_t s = part + 1; s < next; ++s)
      for (int i = tid; i < ct.count * (N + 2); i += 256) p.part_a[(s * p.D + ct.d0) * (N + 2) + i] = 0.f;
  }
}

// Sum of `count` values `stride` apart, eight in flight, in a fixed order.
template <typename T>
__device__ __forceinline__ T strided_sum(const float* p, int64_t count, int64_t stride, T zero) {
  T s[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] = zero;
  int64_t i = 0;
  for (; i + 8 <= count; i += 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] += *reinterpret_cast<const T*>(p + (i + k) * stride);
  }
  for (; i < count; ++i) s[0] += *reinterpret_cast<const T*>(p + i * stride);
  return ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
}

// dB and dC from the channel tiles' sums, four values a thread; the threads behind the
// first `bc` form dA, dDskip and ddt_bias from the segments' and sequences' sums.
template <typename E, int N>
__global__ __launch_bounds__(256) void scan_bwd_finish_kernel(ScanParams p, int tiles, int64_t bc, int64_t parts) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t values = p.rows * p.G * 2 * N;
  if (id < bc) {
    const int64_t i = id * 4;
    if (i >= values) return;
    const f32x4_t s = strided_sum<f32x4_t>(p.part_bc + i, tiles, values, zero4());
    const int64_t rg = i / (2 * N);
    const int k = static_cast<int>(i % (2 * N));
    chunk::store4<E>(static_cast<E*>(k < N ? p.dBm : p.dCm) + rg * N + k % N, s[0], s[1], s[2], s[3]);
    return;
  }
  const int64_t i = id - bc, items = static_cast<int64_t>(p.D) * (N + 2);
  if (i >= items) return;
  const float s = strided_sum<float>(p.part_a + i, parts, items, 0.f);
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

template <typename E, int N, bool GATED>
void launch_main(const ScanParams& p, dim3 grid, hipStream_t s) {
  if (p.seq.cu || p.seq.T % TT != 0)
    hipLaunchKernelGGL((scan_bwd_kernel<E, N, GATED, true>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((scan_bwd_kernel<E, N, GATED, false>), grid, dim3(256), 0, s, p);
}

template <typename E, int N>
hipError_t bwd_t(const ScanParams& p, hipStream_t s) {
  const unsigned tiles = static_cast<unsigned>(scan_tiles(p.D, p.G)), nseq = static_cast<unsigned>(p.nseq);
  if (nseq > 0) {
    if (p.segs > 1)
      hipLaunchKernelGGL((scan_bwd_summary_kernel<E, N>), dim3(tiles, p.segs - 1, nseq), dim3(256), 0, s, p);
    if (p.dz)
      launch_main<E, N, true>(p, dim3(tiles, p.segs, nseq), s);
    else
      launch_main<E, N, false>(p, dim3(tiles, p.segs, nseq), s);
  }
  const int64_t bc = static_cast<int64_t>(blocks_of(p.rows * p.G * N / 2)) * 256;
  hipLaunchKernelGGL((scan_bwd_finish_kernel<E, N>), dim3(blocks_of(bc + static_cast<int64_t>(p.D) * (N + 2))), dim3(256), 0,
                     s, p, static_cast<int>(tiles / p.G), bc, p.parts);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_bwd(const ScanParams& p, int N, bool bf16, hipStream_t s) { GDN_SCAN_DISPATCH(bwd_t) }

}  // namespace gdn
