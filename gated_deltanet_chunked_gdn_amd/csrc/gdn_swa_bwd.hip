// Backward of the window attention on gfx950.  With P from the kept log-sums and
//   delta_i = sum_d do_i o_i,  dP = do v^T,  dS = scale P (dP - delta)
//   dv_j = sum_i P_ij do_i,  dk_j = sum_i dS_ij q_i,  dq_i = sum_j dS_ij k_j
//
// Two kernels form the scores again, each with its own sum in registers, so no sum needs
// an atomic and every result is bit-identical from call to call:
//   * dq: a block of queries over its keys, scores transposed as in the forward; it also
//     forms delta, which the other reads;
//   * dk, dv: a block of keys over the queries whose window holds it, for every query head
//     of its key head; here the scores stand with queries down the accumulator, a key a
//     lane, which makes P and dS the operands of the sums over queries.
// The first tokens are seen by all later queries too: a few keys with long sums.  Their
// part from behind the window is summed by runs of queries (the same kernel, its four waves
// sharing the keys and parting the queries) and joined in order by a last kernel.
//
// Bound by the matrix units and what runs beside them.  4 x 4096 tokens, 16 query heads and 8 key
// heads of 128, window 512, bf16: dq 183 us (109 GFLOP with the edges' tiles whole, 600
// TFLOP/s), dk and dv 217 (137, 630), the first tokens 35 and 7.
// Two waves a SIMD leave 256 registers: dq keeps 48 bytes a lane in scratch there, dk and dv 8.
#include <hip/hip_runtime.h>

#include "gdn_swa_device.h"

namespace gdn {
namespace {

using namespace swa;

// ---------------------------------------------------------------------------- dq

// dq and delta of a block of queries, as the forward's attend.
template <typename Op, int D, int CT, bool CAREFUL>
__device__ __forceinline__ bool dq_block(const SwaParams& p, int64_t bos, int len, int q0, int h, int hk,
                                         typename Op::elem (*Kt)[64 * D], typename Op::elem (*Vt)[64 * D]) {
  using E = typename Op::elem;
  constexpr int KT = 64, QB = 64 * CT, NS = D / Op::kCols, ND = D / 16, KB = Op::kBlocks;
  int thread = threadIdx.x;
  if (CAREFUL) asm volatile("" : "+v"(thread), "+s"(q0), "+s"(h), "+s"(hk));  // no register holds anything for the second time
  const int lane = thread & 63, wave = __builtin_amdgcn_readfirstlane(thread >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int wq0 = q0 + 16 * CT * wave, wq1 = min(wq0 + 16 * CT - 1, len - 1);
  u32x4_t qf[CT][NS], df[CT][NS];
  float lse2[CT], delta[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    const int i = min(wq0 + 16 * t + c, len - 1);
    const int64_t at = (bos + i) * p.Hq + h;
    const E* const row = static_cast<const E*>(p.q) + (bos + i) * p.q_stride + h * D;
    const E* const drow = static_cast<const E*>(p.dout) + at * D;
    const E* const orow = static_cast<const E*>(p.o) + at * D;
    float dot = 0.f;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      qf[t][s] = load_row<Op>(row, s, lane);
      df[t][s] = load_row<Op>(drow, s, lane);
      const u32x4_t of = load_row<Op>(orow, s, lane);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if constexpr (sizeof(E) == 2) {
          dot = fmaf(__uint_as_float(df[t][s][w] << 16), __uint_as_float(of[w] << 16), dot);
          dot = fmaf(__uint_as_float(df[t][s][w] & 0xffff0000u), __uint_as_float(of[w] & 0xffff0000u), dot);
        } else {
          dot = fmaf(__uint_as_float(df[t][s][w]), __uint_as_float(of[w]), dot);
        }
      }
    }
    dot += __shfl_xor(dot, 16, 64);
    dot += __shfl_xor(dot, 32, 64);
    delta[t] = dot;
    lse2[t] = odd_(p.lse[at]) ? __uint_as_float(0x7fc00000u) : p.lse[at] * kLog2e;  // no probability of an infinite sum
  }
  const E* const kb = static_cast<const E*>(p.k) + bos * p.k_stride + hk * D;
  const E* const vb = static_cast<const E*>(p.v) + bos * p.v_stride + hk * D;
  const int win = max(0, q0 - p.W + 1) / KT * KT, last = min(q0 + QB, len) - 1;
  const int nfirst = (min(p.S, win) + KT - 1) / KT, tiles = nfirst + (last - win) / KT + 1;
  auto start = [&](int t) { return t < nfirst ? t * KT : win + (t - nfirst) * KT; };

  f32x4_t acc[ND][CT];
#pragma unroll
  for (int t = 0; t < CT; ++t)
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[d][t] = zero4();
  const float scale2 = p.scale * kLog2e;
  // Where queries see few keys, o is as large as the values and its rounding to bf16 is most of the
  // error of delta (and a third of dq's and dk's): there delta is the sum of P dP, by a pass
  // of its own over the few tiles.
  const bool exact = sizeof(E) == 2 && tiles <= 4;
  const int steps = exact ? 2 * tiles : tiles;
  float own[CT];
#pragma unroll
  for (int u = 0; u < CT; ++u) own[u] = 0.f;
  const Stage<E, D, KT> stage_k(p.k_stride, thread), stage_v(p.v_stride, thread);
  auto fetch = [&](int t) {
    const int j0 = start(t >= tiles ? t - tiles : t);
    stage_k.load(Kt[t & 1], kb + j0 * p.k_stride, len - j0);
    stage_v.load(Vt[t & 1], vb + j0 * p.v_stride, len - j0);
  };
  fetch(0);
  for (int t = 0; t < steps; ++t) {
    const bool sums = exact && t < tiles;  // the pass that forms delta
    const int j0 = start(t >= tiles ? t - tiles : t);
    const E* const Ks = Kt[t & 1];
    const E* const Vs = Vt[t & 1];
    landed();
    __syncthreads();  // and the other buffer is read
    if (t + 1 < steps) fetch(t + 1);
    if (exact && t == tiles) {
#pragma unroll
      for (int u = 0; u < CT; ++u) {
        delta[u] = own[u] + __shfl_xor(own[u], 16, 64);
        delta[u] += __shfl_xor(delta[u], 32, 64);
      }
    }
    if (wq0 >= len) continue;
    // a step of the second product at a time: none seen, all seen, or a mask
#pragma unroll 1
    for (int b0 = 0; b0 < 4; b0 += KB) {
      const int jb = j0 + 16 * b0, je = jb + 16 * KB - 1;
      if (jb > wq1 || (je <= wq0 - p.W && jb >= p.S)) continue;
      const bool whole = je <= wq0 && jb > wq1 - p.W;
      f32x4_t s[KB][CT], dp[KB][CT];
#pragma unroll
      for (int b = 0; b < KB; ++b) {
#pragma unroll
        for (int u = 0; u < CT; ++u) s[b][u] = dp[b][u] = zero4();
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const u32x4_t ka = read_row<Op, D>(Ks, 16 * (b0 + b), n, lane);
          const u32x4_t va = read_row<Op, D>(Vs, 16 * (b0 + b), n, lane);
#pragma unroll
          for (int u = 0; u < CT; ++u) {
            s[b][u] = Op::mma(ka, qf[u][n], s[b][u]);
            dp[b][u] = Op::mma(va, df[u][n], dp[b][u]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < CT; ++u) {
        const float less = sums ? 0.f : delta[u];
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r) s[b][u][r] = exp2_(fmaf(s[b][u][r], scale2, -lse2[u])) * (dp[b][u][r] - less);
      }
      if (!whole) {
        seldom();
#pragma unroll
        for (int u = 0; u < CT; ++u)
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              s[b][u][r] = sees(wq0 + 16 * u + c, jb + 16 * b + 4 * g + r, p.W, p.S) ? s[b][u][r] : 0.f;
      }
      if (sums) {
#pragma unroll
        for (int u = 0; u < CT; ++u)
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) own[u] += s[b][u][r];
        continue;
      }
      u32x4_t sf[CT];
#pragma unroll
      for (int u = 0; u < CT; ++u) {
        const f32x4_t two[2] = {s[0][u], s[KB - 1][u]};
        sf[u] = Op::operand(two);
      }
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        if (CAREFUL) __builtin_amdgcn_sched_barrier(0);  // few registers: one operand after the other
        u32x4_t a = Op::template read_tr<D>(Ks, 16 * b0, 16 * d, lane);
        // who sees such a key has NaN for its probability, unless that is zero
        if (CAREFUL && !whole) a = clean_<E>(a);
#pragma unroll
        for (int u = 0; u < CT; ++u) acc[d][u] = Op::mma(a, sf[u], acc[d][u]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < CT; ++u)
    if (g == 0 && wq0 + 16 * u + c < len) p.delta[(bos + wq0 + 16 * u + c) * p.Hq + h] = delta[u];
  float rest = 0.f;  // NaN, if some sum is not finite
#pragma unroll
  for (int u = 0; u < CT; ++u) {
    const int i = wq0 + 16 * u + c;
    if (i >= len) continue;
    E* const row = static_cast<E*>(p.dq) + ((bos + i) * p.Hq + h) * D;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
#pragma unroll
      for (int r = 0; r < 4; ++r) rest = fmaf(acc[d][u][r], 0.f, rest);
      chunk::store4<E>(row + 16 * d + 4 * g, acc[d][u][0] * p.scale, acc[d][u][1] * p.scale, acc[d][u][2] * p.scale, acc[d][u][3] * p.scale);
    }
  }
  return rest != 0.f;
}

template <typename Op, int D, int CT>
__global__ __launch_bounds__(256, sizeof(typename Op::elem) == 2 ? 2 : 1) void swa_dq_kernel(SwaParams p, SwaWork w) {
  const Item item = item_of(p, w);
  if (item.slot < 0) return;
  const int hk = item.hk, h = hk * w.heads + item.head;
  const Spot at = spot(p, item.slot, 64 * CT);
  const int64_t bos = at.bos;
  const int len = at.len, q0 = at.block * 64 * CT;
  if (q0 >= len) return;

  __shared__ alignas(16) typename Op::elem Kt[2][64 * D], Vt[2][64 * D];
  __shared__ int found;
  if (threadIdx.x == 0) found = 0;
  if (dq_block<Op, D, CT, false>(p, bos, len, q0, h, hk, Kt, Vt)) found = 1;
  __syncthreads();
  if (found) dq_block<Op, D, CT, true>(p, bos, len, q0, h, hk, Kt, Vt);
}

// ---------------------------------------------------------------------------- dk, dv

// What a workgroup's waves hold.
enum Form {
  kKeys,    // 32 keys each, of the queries whose window holds them
  kShared,  // the same 32 keys, and parted queries: where the blocks of 128 keys leave CUs without work
  kFar      // the same 16 first tokens, and parted queries of a run whose window has left them behind
};

template <typename Op, int D, Form FORM>
__global__ __launch_bounds__(256, sizeof(typename Op::elem) == 2 && (D == 64 || FORM == kKeys) ? 2 : 1) void swa_dkv_kernel(SwaParams p, SwaWork w) {
  using E = typename Op::elem;
  constexpr bool FAR = FORM == kFar, PART = FORM != kKeys;  // PART: each wave takes a step of a tile's queries
  constexpr int CT = FAR ? 1 : 2, KW = 16 * CT, KT = PART ? KW : 4 * KW;  // keys of a wave, of the workgroup
  constexpr int KB = Op::kBlocks, NS = D / Op::kCols, ND = D / 16, QT = PART ? 64 * KB : 32;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const Item item = item_of(p, w);
  if (item.slot < 0) return;
  const int group = p.Hq / p.Hk, hk = item.hk;
  const Spot place = spot(p, item.slot, FAR ? p.far : KT);
  const int64_t bos = place.bos;
  const int len = place.len, block = place.block;
  const int k0 = FAR ? KT * blockIdx.z : block * KT, wk0 = PART ? k0 : k0 + KW * wave;
  if (k0 >= len || (FAR && len <= p.W)) return;
  // queries i0 .. i1
  int i0, i1;
  if (FAR) {
    i0 = block * p.far;
    i1 = min(i0 + p.far, len) - 1;
    if (i0 >= len || i1 < k0 + p.W) return;  // a shorter sequence; none of them is so far behind
  } else {
    i0 = k0;
    i1 = min(static_cast<int64_t>(len), static_cast<int64_t>(k0) + KT - 1 + p.W) - 1;
  }

  // the keys stay in LDS, the values in registers: both in registers would leave a SIMD one wave
  __shared__ alignas(16) E Ks[KT * D];
  __shared__ alignas(16) E raw[2][2][QT * D];  // two tiles of queries and of do
  __shared__ alignas(16) float lt[2][QT], dt[2][QT];

  Stage<E, D, KT>(p.k_stride).load(Ks, static_cast<const E*>(p.k) + (bos + k0) * p.k_stride + hk * D, len - k0);
  u32x4_t vf[CT][NS];
#pragma unroll
  for (int u = 0; u < CT; ++u) {
    const int j = min(wk0 + 16 * u + c, len - 1);
    const E* const vrow = static_cast<const E*>(p.v) + (bos + j) * p.v_stride + hk * D;
#pragma unroll
    for (int n = 0; n < NS; ++n) vf[u][n] = load_row<Op>(vrow, n, lane);
  }
  f32x4_t ak[ND][CT], av[ND][CT];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int u = 0; u < CT; ++u) ak[d][u] = av[d][u] = zero4();

  const int tiles = (i1 - i0) / QT + 1, steps = group * tiles;
  const float scale2 = p.scale * kLog2e;
  const int64_t d_stride = static_cast<int64_t>(p.Hq) * D;
  const Stage<E, D, QT> stage_q(p.q_stride), stage_d(d_stride);
  float rl = 0.f, rd = 0.f;
  auto fetch = [&](int step) {
    const int h = hk * group + step / tiles, row = i0 + (step % tiles) * QT;
    stage_q.load(raw[step & 1][0], static_cast<const E*>(p.q) + (bos + row) * p.q_stride + h * D, len - row);
    stage_d.load(raw[step & 1][1], static_cast<const E*>(p.dout) + (bos + row) * d_stride + h * D, len - row);
    if (threadIdx.x < QT) {
      const int64_t at = (bos + min(row + static_cast<int>(threadIdx.x), len - 1)) * p.Hq + h;
      rl = odd_(p.lse[at]) ? __uint_as_float(0x7fc00000u) : p.lse[at] * kLog2e;
      rd = p.delta[at];
    }
  };
  fetch(0);
  for (int step = 0; step < steps; ++step) {
    const int r0 = i0 + (step % tiles) * QT;
    E* const Qs = raw[step & 1][0];
    E* const Ds = raw[step & 1][1];
    const float* const ls = lt[step & 1];
    const float* const dl = dt[step & 1];
    landed();
    if (threadIdx.x < QT) {
      lt[step & 1][threadIdx.x] = rl;
      dt[step & 1][threadIdx.x] = rd;
    }
    __syncthreads();  // and the other buffer is read
    if (step + 1 < steps) fetch(step + 1);
    // Queries, or rows of do, that are not finite, where some key is not seen by them: their
    // lse, or their delta, is not finite either.  Those keys that they see get NaN from it.
    bool strange = false;
    if (FAR || r0 < k0 + KT - 1 || r0 + QT - k0 > p.W) {
      seldom();
#pragma unroll
      for (int i = 0; i < QT; i += 64) strange |= odd_(ls[i + lane % QT]) || odd_(dl[i + lane % QT]);
      strange = __any(strange);  // the same in all waves
      if (strange) {
        clean_part<E, QT * D>(Qs);
        clean_part<E, QT * D>(Ds);
        __syncthreads();
      }
    }
#pragma unroll
    for (int b1 = 0; b1 < (PART ? KB : QT / 16); b1 += KB) {
      const int b0 = PART ? KB * wave : b1;
      const int first = r0 + 16 * b0, end = first + 16 * KB - 1;
      // no query here sees a key of this wave's
      if (wk0 >= len || first >= len || (FAR ? end < wk0 + p.W : end < wk0 || first - (wk0 + KW - 1) >= p.W)) continue;
      const bool whole = !FAR && first >= wk0 + KW - 1 && end - wk0 < p.W && end < len && wk0 + KW - 1 < len;
      f32x4_t s[KB][CT], dp[KB][CT];
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int u = 0; u < CT; ++u) s[b][u] = dp[b][u] = zero4();
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        u32x4_t kf[CT];
#pragma unroll
        for (int u = 0; u < CT; ++u) kf[u] = read_row<Op, D>(Ks, wk0 - k0 + 16 * u, n, lane);
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          const u32x4_t qa = read_row<Op, D>(Qs, 16 * (b0 + b), n, lane);
          const u32x4_t da = read_row<Op, D>(Ds, 16 * (b0 + b), n, lane);
#pragma unroll
          for (int u = 0; u < CT; ++u) {
            s[b][u] = Op::mma(qa, kf[u], s[b][u]);
            dp[b][u] = Op::mma(da, vf[u][n], dp[b][u]);
          }
        }
      }
      u32x4_t pf[CT], sf[CT];
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        const f32x4_t l4 = *reinterpret_cast<const f32x4_t*>(&ls[16 * (b0 + b) + 4 * g]);
        const f32x4_t d4 = *reinterpret_cast<const f32x4_t*>(&dl[16 * (b0 + b) + 4 * g]);
#pragma unroll
        for (int u = 0; u < CT; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            s[b][u][r] = exp2_(fmaf(s[b][u][r], scale2, -l4[r]));
            dp[b][u][r] = s[b][u][r] * (dp[b][u][r] - d4[r]);
          }
      }
      if (!whole) {
        seldom();
#pragma unroll
        for (int u = 0; u < CT; ++u) {
          const int j = wk0 + 16 * u + c;
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int i = first + 16 * b + 4 * g + r;
              const bool ok = i < len && j < len && (FAR ? j < p.S && i - j >= p.W : j <= i && i - j < p.W);
              s[b][u][r] = ok ? s[b][u][r] : 0.f;
              dp[b][u][r] = ok ? dp[b][u][r] : 0.f;
            }
        }
      }
#pragma unroll
      for (int u = 0; u < CT; ++u) {
        const f32x4_t two[2] = {s[0][u], s[KB - 1][u]}, ds[2] = {dp[0][u], dp[KB - 1][u]};
        pf[u] = Op::operand(two);
        sf[u] = Op::operand(ds);
      }
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const u32x4_t da = Op::template read_tr<D>(Ds, 16 * b0, 16 * d, lane);
        const u32x4_t qa = Op::template read_tr<D>(Qs, 16 * b0, 16 * d, lane);
#pragma unroll
        for (int u = 0; u < CT; ++u) {
          av[d][u] = Op::mma(da, pf[u], av[d][u]);
          ak[d][u] = Op::mma(qa, sf[u], ak[d][u]);
        }
      }
    }
    if (strange) {
#pragma unroll 1
      for (int i = r0; i < min(r0 + QT, len); ++i) {
        bool in[CT];
#pragma unroll
        for (int u = 0; u < CT; ++u) {
          const int j = wk0 + 16 * u + c;
          in[u] = j < len && (FAR ? j < p.S && i - j >= p.W : j <= i && i - j < p.W);
        }
        spoil<E, ND, CT>(av, static_cast<const E*>(p.dout) + (bos + i) * d_stride + (hk * group + step / tiles) * D, in, lane);
      }
    }
  }
  if constexpr (PART) {
    // the waves' sums, added in order in LDS and taken over by the first; a lane's values
    // side by side, 16 bytes a lane
    f32x4_t* const sums = reinterpret_cast<f32x4_t*>(&raw[0][0][0]) + lane;
    static_assert(sizeof(raw) >= 2 * ND * CT * 64 * sizeof(f32x4_t), "room for a wave's sums");
    for (int w = 3; w >= 0; --w) {
      __syncthreads();
      if (wave != w) continue;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int u = 0; u < CT; ++u) {
          f32x4_t* const k4 = sums + (2 * (d * CT + u)) * 64;
          f32x4_t* const v4 = k4 + 64;
          if (w < 3) {
            ak[d][u] += *k4;
            av[d][u] += *v4;
          }
          if (w > 0) {
            *k4 = ak[d][u];
            *v4 = av[d][u];
          }
        }
    }
    if (wave) return;
  }
#pragma unroll
  for (int u = 0; u < CT; ++u) {
    const int j = wk0 + 16 * u + c;
    if (j >= len) continue;
    float* part = nullptr;  // of the first tokens
    if (FAR) {
      if (j >= p.S) continue;
      const int64_t slot = bos / p.far + place.n + block;
      part = p.first_far + ((slot * p.Hk + hk) * p.S + j) * 2 * D;
    } else if (j < p.S && len > p.W) {
      part = p.first_win + ((static_cast<int64_t>(place.n) * p.Hk + hk) * p.S + j) * 2 * D;
    }
    if (part) {
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        chunk::store4<float>(part + 16 * d + 4 * g, ak[d][u][0], ak[d][u][1], ak[d][u][2], ak[d][u][3]);
        chunk::store4<float>(part + D + 16 * d + 4 * g, av[d][u][0], av[d][u][1], av[d][u][2], av[d][u][3]);
      }
    } else {
      const int64_t at = ((bos + j) * p.Hk + hk) * D;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        chunk::store4<E>(static_cast<E*>(p.dk) + at + 16 * d + 4 * g, ak[d][u][0] * p.scale, ak[d][u][1] * p.scale, ak[d][u][2] * p.scale,
                         ak[d][u][3] * p.scale);
        chunk::store4<E>(static_cast<E*>(p.dv) + at + 16 * d + 4 * g, av[d][u][0], av[d][u][1], av[d][u][2], av[d][u][3]);
      }
    }
  }
}

// The first tokens' dk and dv: the sums from inside the window, then those of the runs in order.
template <typename E, int D>
__global__ __launch_bounds__(2 * D) void swa_first_kernel(SwaParams p) {
  const int j = blockIdx.x / p.Hk, hk = blockIdx.x % p.Hk, n = blockIdx.y, x = threadIdx.x;
  int64_t bos, len;
  chunk::seq_range(p.seq, n, bos, len);
  if (len <= p.W || j >= len) return;
  float sum = p.first_win[((static_cast<int64_t>(n) * p.Hk + hk) * p.S + j) * 2 * D + x];
  const int64_t slot = bos / p.far + n, runs = (len + p.far - 1) / p.far;
  // as in the kernel above: the keys' block of 16 says which runs were formed
  for (int64_t r = 0; r < runs; ++r)
    if (min((r + 1) * p.far, len) - 1 >= (j & ~15) + p.W) sum += p.first_far[(((slot + r) * p.Hk + hk) * p.S + j) * 2 * D + x];
  const int64_t at = ((bos + j) * p.Hk + hk) * D;
  if (x < D)
    IoT<E>::st(static_cast<E*>(p.dk) + at + x, sum * p.scale);
  else
    IoT<E>::st(static_cast<E*>(p.dv) + at + x - D, sum);
}

template <typename Op, int D, int CT, Form FORM>
hipError_t launch_c(const SwaParams& p, hipStream_t s) {
  SwaGrid g = swa_grid(p, 64 * CT, p.Hq / p.Hk);
  hipLaunchKernelGGL((swa_dq_kernel<Op, D, CT>), g.grid, dim3(256), 0, s, p, g.work);
  g = swa_grid(p, FORM == kKeys ? kSwaKeys : 32, 1);
  hipLaunchKernelGGL((swa_dkv_kernel<Op, D, FORM>), g.grid, dim3(256), 0, s, p, g.work);
  if (p.S > 0) {
    g = swa_grid(p, p.far, 1, (p.S + 15) / 16);
    hipLaunchKernelGGL((swa_dkv_kernel<Op, D, kFar>), g.grid, dim3(256), 0, s, p, g.work);
    hipLaunchKernelGGL((swa_first_kernel<typename Op::elem, D>), dim3(static_cast<unsigned>(p.S * p.Hk), static_cast<unsigned>(p.N)), dim3(2 * D), 0,
                       s, p);
  }
  return hipGetLastError();
}
template <typename Op, int D>
hipError_t launch_t(const SwaParams& p, hipStream_t s) {
  if (p.few) return p.few_keys ? launch_c<Op, D, 1, kShared>(p, s) : launch_c<Op, D, 1, kKeys>(p, s);
  return p.few_keys ? launch_c<Op, D, 2, kShared>(p, s) : launch_c<Op, D, 2, kKeys>(p, s);
}

}  // namespace

hipError_t launch_swa_bwd(const SwaParams& p, int D, bool bf16, hipStream_t s) {
  if (bf16) return D == 64 ? launch_t<MmaBf16, 64>(p, s) : launch_t<MmaBf16, 128>(p, s);
  return D == 64 ? launch_t<MmaF32, 64>(p, s) : launch_t<MmaF32, 128>(p, s);
}

}  // namespace gdn
