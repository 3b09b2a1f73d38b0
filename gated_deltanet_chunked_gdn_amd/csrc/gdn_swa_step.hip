// Window attention over a cache, on gfx950: a single token of every sequence, and the
// filling of the cache from a prompt.
//
// The cache of a sequence has S slots for its first tokens and a ring of W behind them:
// token j >= S stands in slot S + (j - S) mod W.  After any number of tokens the slots that
// have been written hold exactly the keys that the next query sees, so the step attends to
// all of them and takes no mask but their count.
//
// Bound by the cache's bytes: 64 sequences of 4100 slots, 4 key heads of 128, bf16: 504 MB in 98 to
// 101 us, 5.1 TB/s, as a copy (4 us of it the product that keeps the probabilities' lower bits).  The query heads of a key head (up to 16) are the columns of
// one 16x16 product, so every key and value is read once for all of them; keys go from
// memory into the operand, values through a tile in LDS of the wave's own, so the waves of a
// workgroup meet only at the end.  Where the sequences and key heads are few, the slots are parted
// into runs, joined by a second kernel in order.
#include <hip/hip_runtime.h>

#include "gdn_swa_device.h"

namespace gdn {
namespace {

using namespace swa;

template <typename Op, int D, bool SPLIT>
__global__ __launch_bounds__(256, 2) void swa_step_kernel(SwaParams p) {
  using E = typename Op::elem;
  using T = Tile<E, D>;
  constexpr int NS = D / Op::kCols, ND = D / 16, KB = Op::kBlocks, NB = KB;
  constexpr int kWave = 16 * NB;  // slots that a wave takes at a time: a step of the second product
  constexpr int kRows = 64 / T::kPieces, kN = kWave / kRows;  // rows that a wave stages at once
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int n = blockIdx.z, hk = blockIdx.y % p.Hk, group = p.Hq / p.Hk, h0 = hk * group + blockIdx.y / p.Hk * 16;
  const int heads = min(16, (hk + 1) * group - h0);  // query heads of this workgroup
  const int before = p.lens[n], W = p.slots - p.S;
  const int count = before < 0 ? 0 : min(before, p.slots - 1) + 1;
  const int from = blockIdx.x * p.run, to = min(count, from + p.run);
  const int now = before < p.S ? before : p.S + (before - p.S) % W;  // the new token's slot

  static_assert(kWave * sizeof(E) == 16 * sizeof(float), "a wave's tile of values and its sums take the same room");
  __shared__ alignas(16) char raw[4 * 16 * D * sizeof(float)];  // values' tiles, then the waves' sums
  __shared__ float tops[4][16], sums[4][16];
  E* const Vs = reinterpret_cast<E*>(raw) + wave * kWave * D;

  const int64_t row = static_cast<int64_t>(p.Hk) * D;
  const E* const kb = static_cast<const E*>(p.kc) + static_cast<int64_t>(n) * p.slots * row + hk * D;
  const E* const vb = static_cast<const E*>(p.vc) + static_cast<int64_t>(n) * p.slots * row + hk * D;
  const E* const kn = static_cast<const E*>(p.k) + n * p.k_stride + hk * D;
  const E* const vn = static_cast<const E*>(p.v) + n * p.v_stride + hk * D;

  u32x4_t qf[NS];
  const E* const qrow = static_cast<const E*>(p.q) + n * p.q_stride + (h0 + min(c, heads - 1)) * D;
#pragma unroll
  for (int s = 0; s < NS; ++s) qf[s] = load_row<Op>(qrow, s, lane);

  f32x4_t acc[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) acc[d] = zero4();
  float top = -INFINITY, sum = 0.f;
  const float scale2 = p.scale * kLog2e;
  for (int j0 = from + kWave * wave; j0 < to; j0 += 4 * kWave) {
    u32x4_t kf[NB][NS], w[kN];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int j = min(j0 + 16 * b + c, to - 1);
      const E* const krow = j == now ? kn : kb + j * row;
#pragma unroll
      for (int s = 0; s < NS; ++s) kf[b][s] = load_row<Op>(krow, s, lane);
    }
    const int piece = lane % T::kPieces, first = lane / T::kPieces;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int j = j0 + first + i * kRows;
      const E* const vrow = j == now ? vn : vb + min(j, to - 1) * row;
      w[i] = *reinterpret_cast<const u32x4_t*>(vrow + piece * T::kEpp);
      if (j >= to) w[i] = u32x4_t(0u);
    }
    f32x4_t s[NB];
    float high = -INFINITY;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      s[b] = zero4();
#pragma unroll
      for (int m = 0; m < NS; ++m) s[b] = Op::mma(kf[b][m], qf[m], s[b]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[b][r] = j0 + 16 * b + 4 * g + r < to ? s[b][r] * scale2 : -INFINITY;
        high = fmaxf(high, s[b][r]);
      }
    }
    high = fmaxf(high, __shfl_xor(high, 16, 64));
    high = fmaxf(high, __shfl_xor(high, 32, 64));
    const float most = fmaxf(top, high), base = most == -INFINITY ? 0.f : most, fade = exp2_(top - base);
    top = most;
    sum *= fade;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[b][r] = exp2_(s[b][r] - base);
        sum += s[b][r];
      }
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[d] *= fade;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < kN; ++i) *reinterpret_cast<u32x4_t*>(Vs + T::at(first + i * kRows, piece)) = w[i];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int b = 0; b < NB; b += KB) {
      const f32x4_t two[2] = {s[b], s[b + KB - 1]};
      const u32x4_t pf = Op::operand(two);
      u32x4_t rest;  // the matrix units wait for the cache: a second product keeps 16 bits of each probability
      if constexpr (sizeof(E) == 2) rest = Op::rest(two, pf);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const u32x4_t vt = Op::template read_tr<D>(Vs, 16 * b, 16 * d, lane);
        acc[d] = Op::mma(vt, pf, acc[d]);
        if constexpr (sizeof(E) == 2) acc[d] = Op::mma(vt, rest, acc[d]);
      }
    }
  }
  sum += __shfl_xor(sum, 16, 64);
  sum += __shfl_xor(sum, 32, 64);
  if (g == 0) {
    tops[wave][c] = top;
    sums[wave][c] = sum;
  }
  __syncthreads();  // the values' tiles are read
  // the new token's row; nobody reads that slot of the cache
  if (to > from && now >= from && now < to && blockIdx.y < p.Hk && threadIdx.x < 2 * T::kPieces) {
    const bool val = threadIdx.x >= T::kPieces;
    const int at = (threadIdx.x % T::kPieces) * T::kEpp;
    E* const dst = static_cast<E*>(val ? p.vc : p.kc) + (static_cast<int64_t>(n) * p.slots + now) * row + hk * D + at;
    *reinterpret_cast<u32x4_t*>(dst) = *reinterpret_cast<const u32x4_t*>((val ? vn : kn) + at);
  }
  float most = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) most = fmaxf(most, tops[i][c]);
  const float base = most == -INFINITY ? 0.f : most, mine = exp2_(top - base);
  float* const os = reinterpret_cast<float*>(raw) + (wave * 16 + c) * D;  // [wave][head][D], pieces swizzled by the head
#pragma unroll
  for (int d = 0; d < ND; ++d)
    *reinterpret_cast<f32x4_t*>(os + (((4 * d + g) ^ c) * 4)) = acc[d] * mine;
  __syncthreads();
  // D / 4 pieces of 16 heads
#pragma unroll
  for (int i = 0; i < 16 * D / 4 / 256; ++i) {
    const int at = threadIdx.x + 256 * i, head = at / (D / 4), piece = at % (D / 4);
    if (head >= heads) continue;
    f32x4_t o = zero4();
    float total = 0.f, high = -INFINITY;
#pragma unroll
    for (int k = 0; k < 4; ++k) high = fmaxf(high, tops[k][head]);
    const float zero = high == -INFINITY ? 0.f : high;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o += *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(raw) + (k * 16 + head) * D + ((piece ^ head) * 4));
      total = fmaf(sums[k][head], exp2_(tops[k][head] - zero), total);
    }
    const int64_t out = static_cast<int64_t>(n) * p.Hq + h0 + head, all = static_cast<int64_t>(p.N) * p.Hq;
    if constexpr (SPLIT) {
      const int64_t at_part = blockIdx.x * all + out;
      if (piece == 0) *reinterpret_cast<float2*>(p.part + 2 * at_part) = float2{high, total};
      *reinterpret_cast<f32x4_t*>(p.part + 2 * all * p.splits + at_part * D + 4 * piece) = o;
    } else {
      const float inv = before < 0 ? 0.f : 1.f / total;
      chunk::store4<E>(static_cast<E*>(p.o) + out * D + 4 * piece, o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
    }
  }
}

// The runs' sums joined in order, a head a workgroup: four parts of them side by side, then
// those.  A lane takes a run's maximum and sum, 64 runs at a time, and a thread a column of the
// values, one run after another.  (One part took 7 us longer over 118 runs.)
constexpr int kJoin = 4;
template <typename E, int D>
__global__ __launch_bounds__(kJoin * D) void swa_join_kernel(SwaParams p) {
  __shared__ float tops[kJoin], sums[kJoin], cols[kJoin][D];
  const int n = blockIdx.y, part = threadIdx.x / D, x = threadIdx.x % D, lane = x & 63;
  const int64_t out = static_cast<int64_t>(n) * p.Hq + blockIdx.x, all = static_cast<int64_t>(p.N) * p.Hq;
  const float* const vals = p.part + 2 * all * p.splits + out * D + x;
  const int before = p.lens[n];
  const int count = before < 0 ? 0 : min(before, p.slots - 1) + 1, runs = (count + p.run - 1) / p.run;
  const int each = (runs + kJoin - 1) / kJoin, end = min(runs, (part + 1) * each);
  float high = -INFINITY, total = 0.f, o = 0.f;
  for (int s0 = part * each; s0 < end; s0 += 64) {
    const int many = min(end - s0, 64);
    const float2 t = lane < many ? *reinterpret_cast<const float2*>(p.part + 2 * ((s0 + lane) * all + out)) : float2{-INFINITY, 0.f};
    float m = t.x;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    const float now = fmaxf(high, m), base = now == -INFINITY ? 0.f : now, fade = exp2_(high - base);
    high = now;
    const float f = exp2_(t.x - base);
    total = fmaf(total, fade, wave_sum(t.y * f));
    o *= fade;
    for (int s = 0; s < many; ++s) o = fmaf(vals[(s0 + s) * all * D], __shfl(f, s, 64), o);
  }
  if (x == 0) {
    tops[part] = high;
    sums[part] = total;
  }
  cols[part][x] = o;
  __syncthreads();
  if (part) return;
  float most = tops[0];
#pragma unroll
  for (int i = 1; i < kJoin; ++i) most = fmaxf(most, tops[i]);
  const float base = most == -INFINITY ? 0.f : most;
  total = o = 0.f;
#pragma unroll
  for (int i = 0; i < kJoin; ++i) {
    const float f = exp2_(tops[i] - base);
    total = fmaf(sums[i], f, total);
    o = fmaf(cols[i][x], f, o);
  }
  IoT<E>::st(static_cast<E*>(p.o) + out * D + x, before < 0 ? 0.f : o / total);
}

// ---------------------------------------------------------------------------- cache from a prompt

template <typename E>
__global__ __launch_bounds__(256) void swa_fill_kernel(SwaParams p, int row) {
  constexpr int epp = 16 / static_cast<int>(sizeof(E));
  int64_t bos, len;
  chunk::seq_range(p.seq, blockIdx.y, bos, len);
  const int64_t pieces = row / epp, at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t slot = at / pieces, x = (at - slot * pieces) * epp;
  if (slot >= p.slots) return;
  const int64_t W = p.slots - p.S;
  int64_t token = slot;
  if (slot >= p.S) {
    // the last of the tokens behind the first S that fall on the slot
    const int64_t last = len - 1 - p.S, place = slot - p.S;
    if (last < place) return;
    token = p.S + last - (last - place) % W;
  } else if (slot >= len) {
    return;
  }
  const int64_t to = (static_cast<int64_t>(blockIdx.y) * p.slots + slot) * row + x;
  *reinterpret_cast<u32x4_t*>(static_cast<E*>(p.kc) + to) =
      *reinterpret_cast<const u32x4_t*>(static_cast<const E*>(p.k) + (bos + token) * p.k_stride + x);
  *reinterpret_cast<u32x4_t*>(static_cast<E*>(p.vc) + to) =
      *reinterpret_cast<const u32x4_t*>(static_cast<const E*>(p.v) + (bos + token) * p.v_stride + x);
}

template <typename Op, int D>
hipError_t launch_t(const SwaParams& p, hipStream_t s) {
  const int passes = (p.Hq / p.Hk + 15) / 16;
  const dim3 grid(static_cast<unsigned>(p.splits), static_cast<unsigned>(p.Hk * passes), static_cast<unsigned>(p.N));
  if (p.splits == 1) {
    hipLaunchKernelGGL((swa_step_kernel<Op, D, false>), grid, dim3(256), 0, s, p);
  } else {
    hipLaunchKernelGGL((swa_step_kernel<Op, D, true>), grid, dim3(256), 0, s, p);
    hipLaunchKernelGGL((swa_join_kernel<typename Op::elem, D>), dim3(static_cast<unsigned>(p.Hq), static_cast<unsigned>(p.N)), dim3(kJoin * D), 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_swa_step(const SwaParams& p, int D, bool bf16, hipStream_t s) {
  if (bf16) return D == 64 ? launch_t<MmaBf16, 64>(p, s) : launch_t<MmaBf16, 128>(p, s);
  return D == 64 ? launch_t<MmaF32, 64>(p, s) : launch_t<MmaF32, 128>(p, s);
}

hipError_t launch_swa_fill(const SwaParams& p, int D, bool bf16, hipStream_t s) {
  const int row = p.Hk * D;
  const int64_t threads = static_cast<int64_t>(p.slots) * (row / (bf16 ? 8 : 4));
  const dim3 grid(static_cast<unsigned>((threads + 255) / 256), static_cast<unsigned>(p.N));
  if (bf16)
    hipLaunchKernelGGL(swa_fill_kernel<uint16_t>, grid, dim3(256), 0, s, p, row);
  else
    hipLaunchKernelGGL(swa_fill_kernel<float>, grid, dim3(256), 0, s, p, row);
  return hipGetLastError();
}

}  // namespace gdn
