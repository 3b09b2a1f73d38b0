// Causal attention over a sliding window whose first tokens stay visible, forward, on
// gfx950:  o_i = sum_j p_ij v_j,  p_i = softmax over the visible j of scale q_i . k_j.
//
// One pass over the keys that a block of queries sees, with the running maximum and sum of
// the softmax (in base 2, fp32).  A workgroup holds 128 queries of a head, 32 a wave (half
// as many where that leaves CUs without work); keys
// and values come in tiles of 64 rows through LDS, loaded while the tile before is worked
// on.  Scores are formed transposed (keys down the accumulator, a query a lane), so the
// softmax runs inside lanes but for two exchanges of the maximum, and the probabilities are
// the operand of the second product as they stand.  Tiles that all of a wave's queries see
// whole take no mask, those that none sees no product.
//
// Bound by the matrix units and what runs beside them.  2 x 4096 tokens, 16 heads of 128, window
// 1024, bf16: 96 us, 60 GFLOP (70 with the edges' tiles whole) at 630 (730) TFLOP/s (a large
// product: 1320), matrix units busy 40 % of the cycles; taking away the loads, the reads from LDS or the exponentials gains 3 to 10 % each.
#include <hip/hip_runtime.h>

#include "gdn_swa_device.h"

namespace gdn {
namespace {

using namespace swa;

// The outputs of a block of queries q0 .. (CT 16-query columns of a wave: two or, where that
// leaves CUs without work, one); whether this lane's sums are not all finite.  CAREFUL: values
// that are not finite reach the queries that see them alone.
template <typename Op, int D, int CT, bool CAREFUL>
__device__ __forceinline__ bool attend(const SwaParams& p, int64_t bos, int len, int q0, int h, int hk,
                                       typename Op::elem (*Kt)[64 * D], typename Op::elem (*Vt)[64 * D], int* odd) {
  using E = typename Op::elem;
  constexpr int KT = 64, QB = 64 * CT, NS = D / Op::kCols, NR = 4 / Op::kBlocks, ND = D / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int wq0 = q0 + 16 * CT * wave, wq1 = min(wq0 + 16 * CT - 1, len - 1);  // this wave's queries; none if wq0 >= len
  u32x4_t qf[CT][NS];
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    const int i = min(wq0 + 16 * t + c, len - 1);
    const E* const row = static_cast<const E*>(p.q) + (bos + i) * p.q_stride + h * D;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      qf[t][s] = load_row<Op>(row, s, lane);
      // a negative scale turns the queries, so that the largest product has the largest score
      if (p.scale < 0.f) qf[t][s] ^= u32x4_t(sizeof(E) == 2 ? 0x80008000u : 0x80000000u);
    }
  }
  const E* const kb = static_cast<const E*>(p.k) + bos * p.k_stride + hk * D;
  const E* const vb = static_cast<const E*>(p.v) + bos * p.v_stride + hk * D;

  // tiles: the first tokens' as far as they lie before the window's, then the window's
  const int win = max(0, q0 - p.W + 1) / KT * KT, last = min(q0 + QB, len) - 1;
  const int nfirst = (min(p.S, win) + KT - 1) / KT, tiles = nfirst + (last - win) / KT + 1;
  auto start = [&](int t) { return t < nfirst ? t * KT : win + (t - nfirst) * KT; };

  // What the queries do not see of a tile to minus infinity.  Tiles of first tokens lie before
  // every window; of tiles behind the first tokens the window is all.
  auto mask = [&](bool first, int j0, f32x4_t (*to)[CT]) {
    if (first) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool ok = j0 + 16 * b + 4 * g + r < p.S;
#pragma unroll
          for (int u = 0; u < CT; ++u) to[b][u][r] = ok ? to[b][u][r] : -INFINITY;
        }
    } else if (j0 >= p.S) {
#pragma unroll
      for (int u = 0; u < CT; ++u) {
        const int back = wq0 + 16 * u + c - j0 - 4 * g;  // from the lane's first key to the query
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            to[b][u][r] = static_cast<uint32_t>(back - 16 * b - r) < static_cast<uint32_t>(p.W) ? to[b][u][r] : -INFINITY;
      }
    } else {
#pragma unroll
      for (int u = 0; u < CT; ++u)
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            to[b][u][r] = sees(wq0 + 16 * u + c, j0 + 16 * b + 4 * g + r, p.W, p.S) ? to[b][u][r] : -INFINITY;
    }
  };

  f32x4_t acc[ND][CT];
  float top[CT], sum[CT];  // the exponents' base, in base 2, and the sum of this lane's keys
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    top[t] = -INFINITY;
    sum[t] = 0.f;
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[d][t] = zero4();
  }
  const float scale2 = fmaxf(fabsf(p.scale) * kLog2e, 1e-37f);  // not zero: -inf stays what is masked
  const Stage<E, D, KT> stage_k(p.k_stride), stage_v(p.v_stride);
  auto fetch_k = [&](int t) {
    if (t < tiles) stage_k.load(Kt[t & 1], kb + start(t) * p.k_stride, len - start(t));
  };
  auto fetch_v = [&](int t) {
    if (t < tiles) stage_v.load(Vt[t & 1], vb + start(t) * p.v_stride, len - start(t));
  };
  // some query of this wave's sees a key of the tile
  auto some = [&](int t) {
    const int j0 = start(t);
    return t < tiles && wq0 < len && j0 <= wq1 && (j0 + KT - 1 > wq0 - p.W || j0 < p.S);
  };
  f32x4_t s[4][CT], next[4][CT];
  auto scores = [&](int t, f32x4_t (*to)[CT]) {
    const E* const Ks = Kt[t & 1];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
#pragma unroll
      for (int u = 0; u < CT; ++u) to[b][u] = zero4();
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const u32x4_t a = read_row<Op, D>(Ks, 16 * b, n, lane);
#pragma unroll
        for (int u = 0; u < CT; ++u) to[b][u] = Op::mma(a, qf[u][n], to[b][u]);
      }
    }
  };
  auto exponentials = [&]() {
#pragma unroll
    for (int u = 0; u < CT; ++u) {
      const float base = top[u] == -INFINITY ? 0.f : top[u];  // nothing seen yet
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          s[b][u][r] = exp2_(fmaf(s[b][u][r], scale2, -base));
          sum[u] += s[b][u][r];
        }
    }
  };
  // The scores are formed a tile ahead, so that their products run beside the exponentials of
  // the tile before; keys are loaded a tile ahead of the values for that.
  if (CAREFUL && threadIdx.x == 0) odd[0] = 0;
  fetch_k(0);
  landed();
  __syncthreads();
  fetch_v(0);
  fetch_k(1);
  bool now = some(0);
  if (now) scores(0, s);
  for (int t = 0; t < tiles; ++t) {
    const int j0 = start(t);
    landed();
    __syncthreads();  // values of this tile and keys of the next are there, those of the last two read
    fetch_v(t + 1);
    fetch_k(t + 2);
    const bool then = some(t + 1);
    bool strange = false;
    if constexpr (CAREFUL) {
      if (threadIdx.x == 0) odd[(t + 1) & 1] = 0;
      if (j0 + KT - 1 > q0 || j0 <= last - p.W) {  // some query does not see all of it
        if (odd_part<E, KT * D>(Vt[t & 1])) odd[t & 1] = 1;
        __syncthreads();
        strange = odd[t & 1] != 0;
        if (strange) {
          clean_part<E, KT * D>(Vt[t & 1]);
          __syncthreads();
        }
      }
    }
    if (now) {
      if (!(j0 + KT - 1 <= wq0 && j0 > wq1 - p.W)) {
        seldom();
        mask(t < nfirst, j0, s);
      }
      float high[CT];
      bool rise = false;
#pragma unroll
      for (int u = 0; u < CT; ++u) {
        high[u] = -INFINITY;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r) high[u] = fmaxf(high[u], s[b][u][r]);
        // a score may pass the base by 2^8 before all that has been summed is brought to a new
        // one: powers of two change no rounding, and after a few tiles no base moves
        rise |= high[u] * scale2 > top[u] + 8.f;
      }
      if (__any(rise)) {
#pragma unroll
        for (int u = 0; u < CT; ++u) {
          float m = fmaxf(high[u], __shfl_xor(high[u], 16, 64));
          m = fmaxf(m, __shfl_xor(m, 32, 64));
          const float base = fmaxf(top[u], m * scale2);
          const float fade = base == -INFINITY ? 1.f : exp2_(top[u] - base);
          top[u] = base;
          sum[u] *= fade;
#pragma unroll
          for (int d = 0; d < ND; ++d) acc[d][u] *= fade;
        }
      }
      scores(t + 1, next);  // whether there is one or not: no branch between these and the exponentials
      exponentials();
      const E* const Vs = Vt[t & 1];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        u32x4_t pf[CT];
#pragma unroll
        for (int u = 0; u < CT; ++u) {
          const f32x4_t two[2] = {s[n * Op::kBlocks][u], s[n * Op::kBlocks + Op::kBlocks - 1][u]};
          pf[u] = Op::operand(two);
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          const u32x4_t a = Op::template read_tr<D>(Vs, n * 16 * Op::kBlocks, 16 * d, lane);
#pragma unroll
          for (int u = 0; u < CT; ++u) acc[d][u] = Op::mma(a, pf[u], acc[d][u]);
        }
      }
      if (CAREFUL && strange) {
#pragma unroll 1
        for (int j = j0; j < min(j0 + KT, len); ++j) {
          bool in[CT];
#pragma unroll
          for (int u = 0; u < CT; ++u) in[u] = sees(wq0 + 16 * u + c, j, p.W, p.S);
          spoil<E, ND, CT>(acc, vb + j * p.v_stride, in, lane);
        }
      }
    } else if (then) {
      scores(t + 1, next);
    }
    now = then;
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int u = 0; u < CT; ++u) s[b][u] = next[b][u];
  }
  float rest = 0.f;  // NaN, if some sum is not finite
#pragma unroll
  for (int u = 0; u < CT; ++u) {
    const int i = wq0 + 16 * u + c;
    float total = sum[u];
    total += __shfl_xor(total, 16, 64);
    total += __shfl_xor(total, 32, 64);
    if (i >= len) continue;
    const float inv = 1.f / total;
    E* const row = static_cast<E*>(p.o) + ((bos + i) * p.Hq + h) * D;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
#pragma unroll
      for (int r = 0; r < 4; ++r) rest = fmaf(acc[d][u][r], 0.f, rest);
      chunk::store4<E>(row + 16 * d + 4 * g, acc[d][u][0] * inv, acc[d][u][1] * inv, acc[d][u][2] * inv, acc[d][u][3] * inv);
    }
    if (p.lse && g == 0) p.lse[(bos + i) * p.Hq + h] = kLn2 * (top[u] + __builtin_amdgcn_logf(total));
  }
  return rest != 0.f;
}

template <typename Op, int D, int CT>
__global__ __launch_bounds__(256, sizeof(typename Op::elem) == 2 ? 2 : 1) void swa_fwd_kernel(SwaParams p, SwaWork w) {
  const Item item = item_of(p, w);
  if (item.slot < 0) return;
  const int hk = item.hk, h = hk * w.heads + item.head;
  const Spot at = spot(p, item.slot, 64 * CT);
  const int64_t bos = at.bos;
  const int len = at.len, q0 = at.block * 64 * CT;
  if (q0 >= len) return;

  __shared__ alignas(16) typename Op::elem Kt[2][64 * D], Vt[2][64 * D];
  __shared__ int odd[2], found;
  if (threadIdx.x == 0) found = 0;
  // sums that are not finite: once more, with care for those that should be
  if (attend<Op, D, CT, false>(p, bos, len, q0, h, hk, Kt, Vt, odd)) found = 1;
  __syncthreads();
  int again = q0;
  asm volatile("" : "+s"(again));  // nothing of the first time is kept in registers for it
  if (found) attend<Op, D, CT, true>(p, bos, len, again, h, hk, Kt, Vt, odd);
}

template <typename Op, int D, int CT>
hipError_t launch_c(const SwaParams& p, hipStream_t s) {
  const SwaGrid g = swa_grid(p, 64 * CT, p.Hq / p.Hk);
  hipLaunchKernelGGL((swa_fwd_kernel<Op, D, CT>), g.grid, dim3(256), 0, s, p, g.work);
  return hipGetLastError();
}
template <typename Op, int D>
hipError_t launch_t(const SwaParams& p, hipStream_t s) {
  return p.few ? launch_c<Op, D, 1>(p, s) : launch_c<Op, D, 2>(p, s);
}

}  // namespace

hipError_t launch_swa_fwd(const SwaParams& p, int D, bool bf16, hipStream_t s) {
  if (bf16) return D == 64 ? launch_t<MmaBf16, 64>(p, s) : launch_t<MmaBf16, 128>(p, s);
  return D == 64 ? launch_t<MmaF32, 64>(p, s) : launch_t<MmaF32, 128>(p, s);
}

}  // namespace gdn
