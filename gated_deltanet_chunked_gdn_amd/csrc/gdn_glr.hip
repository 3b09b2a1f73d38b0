// The gated linear recurrence on gfx950: per sequence and channel
//
//   la = -c softplus(lam) sigmoid(r_t);  a = exp(la);  m = sqrt(1 - a^2)
//   h <- a h + m sigmoid(i_t) x_t;  y_t = h  or  h silu(z_t)
//
// A linear recurrence composes: a run of tokens takes h to A h + B, with A the product of
// its decays and B its end from zero.  A workgroup holds 32 channels (rows of 64 or 128
// bytes) and walks over its tokens in tiles; a thread takes a run of eight tokens of two or
// four channels, so the tile's runs are composed by lane shifts inside a
// wave and through LDS between waves, and the run is gone through once more from its own
// start.  Inputs are read once, while the tile before is worked on.  Where the channels
// alone are too few workgroups, sequences are cut into segments whose (A, B) come from a
// pass of their own, over the inputs once more.
//
// Backward.  With K_t = dL/dh_t through the later tokens and ds_t = dL/dh_t through y_t,
//   G_t = ds_t + K_t;  K_{t-1} = a_t G_t
// which is the same recurrence from the end; states come from those that the forward keeps
// every eight tokens (1/16 of what it reads, and exact in fp32).  With la times its own
// gradient no quotient grows without bound (m ~ sqrt(-2 la) where la is small):
//   E = G (a la h_{t-1} - a^2 (la / m) sigmoid(i) x)
//   dr = E (1 - sigmoid(r));  dlam = sum_t E sigmoid(lam) / softplus(lam)
//   dx = G m sigmoid(i);  di = G m x sigmoid(i) (1 - sigmoid(i));  dz = dy h silu'(z)
#include <hip/hip_runtime.h>

#include "gdn_hybrid.h"
#include "gdn_layer_device.h"

namespace gdn {
namespace {

using namespace layer;

constexpr int kRun = kGlrRun;
constexpr float kLn2 = 0.6931471805599453f;

// V values of type E as loaded, one vector of 4, 8 or 16 bytes.
template <typename E, int V>
struct Row {
  static constexpr int kWords = V * static_cast<int>(sizeof(E)) / 4;
  typedef uint32_t vec_t __attribute__((ext_vector_type(kWords)));
  vec_t w;
  __device__ __forceinline__ void load(const E* p) { w = *reinterpret_cast<const vec_t*>(p); }
  // through a resource: zeros behind its end, and stores there are dropped
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t byte) {
    if constexpr (kWords == 1)
      w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, byte, 0, 0);
    else
      w = __builtin_bit_cast(vec_t, __builtin_amdgcn_raw_buffer_load_b64(r, byte, 0, 0));
  }
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t byte, const float* f) {
    vec_t v;
#pragma unroll
    for (int i = 0; i < kWords; ++i) v[i] = sizeof(E) == 2 ? pack_bf16x2(f[2 * i], f[2 * i + 1]) : __float_as_uint(f[i]);
    if constexpr (kWords == 1)
      __builtin_amdgcn_raw_buffer_store_b32(v[0], r, byte, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(chunk::u32x2v_t, v), r, byte, 0, 0);
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(E) == 2) {
      const uint32_t x = w[e >> 1];
      return __uint_as_float((e & 1) ? (x & 0xffff0000u) : (x << 16));
    } else {
      return __uint_as_float(w[e]);
    }
  }
  // Hides from the compiler that the values are those of before: what follows forms them again
  // instead of holding on to what was formed from them.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      uint32_t x = w[i];
      asm volatile("" : "+v"(x));
      w[i] = x;
    }
  }
  static __device__ __forceinline__ void store(E* p, const float* f) {
    vec_t v;
#pragma unroll
    for (int i = 0; i < kWords; ++i) v[i] = sizeof(E) == 2 ? pack_bf16x2(f[2 * i], f[2 * i + 1]) : __float_as_uint(f[i]);
    *reinterpret_cast<vec_t*>(p) = v;
  }
};

template <int V>
__device__ __forceinline__ void load_f32(const float* p, bool ok, float* f, float otherwise = 0.f) {
  Row<float, V> v;
  if (ok) v.load(p);
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = ok ? v.get(e) : otherwise;
}

// -c softplus(lam) in log2 units: la = rate sigmoid(r)
__device__ __forceinline__ float rate_(float lam, float c) {
  float sig;
  return -c * softplus_(lam, sig) * kLog2e;
}

// m^2 = 1 - a^2 = 2 a sinh(-la).  Near la = 0 the difference loses what matters, and the
// series of sinh is short (four terms: the fifth is below 2^-26 of the sum for -la <= 1/2);
// beyond, 1 - a^2 is 0.63 and more.
__device__ __forceinline__ float one_minus_square(float la2, float a) {
  const float x = la2 * -kLn2, y = x * x;
  const float s = fmaf(y, fmaf(y, fmaf(y, 2.f / 5040.f, 2.f / 120.f), 2.f / 6.f), 2.f);
  return x < 0.5f ? a * x * s : fmaf(-a, a, 1.f);
}
__device__ __forceinline__ float root_(float x) { return __builtin_amdgcn_sqrtf(x); }

// Tile of 8 XCDs in turn: workgroups x, x + 8, ... share one, so neighbouring channels,
// which share cache lines, go to one L2.
__device__ __forceinline__ int xcd_tile(int x, int tiles) { return (x & 7) * ((tiles + 7) / 8) + (x >> 3); }

// Where a workgroup's thread stands: lanes of a row, runs of a wave, its own run.
template <int V, int NW>
struct Place {
  static constexpr int kLanes = kGlrTile / V;       // lanes of a row
  static constexpr int kRuns = 64 / kLanes;         // runs of a wave
  static constexpr int kTokens = kRuns * kRun * NW; // tokens of a tile
  int lane, wave, run, ch;                          // ch: first channel in the tile's 32
  __device__ __forceinline__ Place() {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    run = lane / kLanes;
    ch = (lane % kLanes) * V;
  }
  __device__ __forceinline__ int token() const { return (wave * kRuns + run) * kRun; }
};

// A tile's rows of one tensor, as a resource that ends with the segment, which is `left` rows
// off: at most 2^30 bytes (512 rows of bf16 or 256 of fp32, of 2^20 values).
template <typename E, int ROWS>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_of(const void* base, int64_t row, int64_t left, int C) {
  static_assert(ROWS * sizeof(E) <= 1024, "2^30 bytes");
  const int64_t rows = min(left, static_cast<int64_t>(ROWS));
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(static_cast<const E*>(base) + row * C), 0,
                                           static_cast<int>(static_cast<uint32_t>(rows) * C * sizeof(E)), 0x00020000);
}

// (A, B) of the runs before this lane's in the wave, (1, 0) in front of the first; `A`, `B`
// become the wave's up to and with this lane.
template <int V, int LANES>
__device__ __forceinline__ void scan_runs(float* A, float* B, float* eA, float* eB, int lane) {
#pragma unroll
  for (int off = LANES; off < 64; off <<= 1) {
    const bool in = lane >= off;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float pa = __shfl_up(A[e], off, 64), pb = __shfl_up(B[e], off, 64);
      if (in) {
        B[e] = fmaf(A[e], pb, B[e]);
        A[e] *= pa;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float pa = __shfl_up(A[e], LANES, 64), pb = __shfl_up(B[e], LANES, 64);
    eA[e] = lane >= LANES ? pa : 1.f;
    eB[e] = lane >= LANES ? pb : 0.f;
  }
}
// The same from the end: runs behind this lane's.
template <int V, int LANES>
__device__ __forceinline__ void scan_runs_back(float* A, float* B, float* eA, float* eB, int lane) {
#pragma unroll
  for (int off = LANES; off < 64; off <<= 1) {
    const bool in = lane + off < 64;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float pa = __shfl_down(A[e], off, 64), pb = __shfl_down(B[e], off, 64);
      if (in) {
        B[e] = fmaf(A[e], pb, B[e]);
        A[e] *= pa;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float pa = __shfl_down(A[e], LANES, 64), pb = __shfl_down(B[e], LANES, 64);
    eA[e] = lane + LANES < 64 ? pa : 1.f;
    eB[e] = lane + LANES < 64 ? pb : 0.f;
  }
}

// ---------------------------------------------------------------------------- forward

// Z: there is a gate.  SUM: the segments' (A, B) alone.
template <typename E, int V, int NW, bool Z, bool SUM>
__global__ __launch_bounds__(64 * NW) void glr_fwd_kernel(GlrParams p, int tiles) {
  using P = Place<V, NW>;
  const P at;
  const int tile = xcd_tile(blockIdx.x, tiles);
  if (tile >= tiles) return;
  const int n = blockIdx.y, s = blockIdx.z;
  int64_t bos, len;
  chunk::seq_range(p.seq, n, bos, len);
  const int64_t t_begin = s * p.seg_len, t_end = min(len, t_begin + p.seg_len);
  // a segment that starts behind its sequence has nothing to do (the first keeps an empty
  // sequence's state), and nothing follows the last one that needs its (A, B)
  if (s > 0 && t_begin >= len) return;
  if (SUM && t_begin + p.seg_len >= len) return;
  const bool chan = tile * kGlrTile + at.ch < p.C;  // whole vectors: C is a multiple of 8
  const int d = chan ? tile * kGlrTile + at.ch : 0;
  __shared__ alignas(16) float pair[2][NW][2][kGlrTile];

  float rate[V], carry[V];
  load_f32<V>(p.lam + d, true, rate);
#pragma unroll
  for (int e = 0; e < V; ++e) rate[e] = rate_(rate[e], p.c);
  load_f32<V>(p.h0 + static_cast<int64_t>(n) * p.C + d, p.h0 != nullptr && !SUM, carry);
  const int64_t slot = bos / p.seg_len + n;
  float prod[V];  // SUM: the product of all decays so far
#pragma unroll
  for (int e = 0; e < V; ++e) prod[e] = 1.f;
  if (!SUM) {
    for (int j = 0; j < s; ++j) {
      float a[V], b[V];
      load_f32<V>(p.seg + (slot + j) * 2 * p.C + d, true, a);
      load_f32<V>(p.seg + ((slot + j) * 2 + 1) * p.C + d, true, b);
#pragma unroll
      for (int e = 0; e < V; ++e) carry[e] = fmaf(a[e], carry[e], b[e]);
    }
  }

  // offset of this thread's run in a tile; of channels behind the last, behind every tile's end
  const uint32_t step = static_cast<uint32_t>(p.C) * sizeof(E);
  const uint32_t first = chan ? static_cast<uint32_t>(at.token()) * step + static_cast<uint32_t>(d * sizeof(E)) : 0x7ffffff0u - kRun * step;
  Row<E, V> rx[kRun], rr[kRun], ri[kRun], rz[kRun];
  auto fetch = [&](int64_t t0) {
    const __amdgpu_buffer_rsrc_t x = tile_of<E, P::kTokens>(p.x, bos + t0, t_end - t0, p.C), r = tile_of<E, P::kTokens>(p.r, bos + t0, t_end - t0, p.C),
                                 gi = tile_of<E, P::kTokens>(p.i, bos + t0, t_end - t0, p.C);
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      rr[j].load(r, first + j * step);
      ri[j].load(gi, first + j * step);
      rx[j].load(x, first + j * step);
    }
    if constexpr (Z) {
      const __amdgpu_buffer_rsrc_t z = tile_of<E, P::kTokens>(p.z, bos + t0, t_end - t0, p.C);
#pragma unroll
      for (int j = 0; j < kRun; ++j) rz[j].load(z, first + j * step);
    }
  };
  // The pass for the sums goes from the segment's end to its start, so that the cache that all
  // XCDs share holds the first of what the next pass reads.
  const int64_t count = (t_end - t_begin + P::kTokens - 1) / P::kTokens;
  if (count > 0) fetch(SUM ? t_begin + (count - 1) * P::kTokens : t_begin);
  int buf = 0;
  for (int64_t k = 0; k < count; ++k, buf ^= 1) {
    const int64_t t0 = t_begin + (SUM ? count - 1 - k : k) * P::kTokens;
    const int have = static_cast<int>(min(t_end - t0, static_cast<int64_t>(512))) - at.token();  // tokens of the run and behind it
    Row<E, V> cx[kRun], cr[kRun], ci[kRun], cz[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      cx[j] = rx[j];
      cr[j] = rr[j];
      ci[j] = ri[j];
      if constexpr (Z) cz[j] = rz[j];
    }
    if (k + 1 < count) fetch(SUM ? t0 - P::kTokens : t0 + P::kTokens);
    float a[kRun][V], b[kRun][V];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float la2 = rate[e] * sigmoid_(cr[j].get(e));
        const float decay = exp2_(la2);
        a[j][e] = decay;
        b[j][e] = root_(one_minus_square(la2, decay)) * sigmoid_(ci[j].get(e)) * cx[j].get(e);
      }
    }
    if (t_end - t0 < P::kTokens) {  // behind the end a token changes nothing (b is zero, as x there)
#pragma unroll
      for (int j = 0; j < kRun; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) a[j][e] = j < have ? a[j][e] : 1.f;
    }
    float A[V], B[V], eA[V], eB[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      A[e] = a[0][e];
      B[e] = b[0][e];
#pragma unroll
      for (int j = 1; j < kRun; ++j) {
        B[e] = fmaf(a[j][e], B[e], b[j][e]);
        A[e] *= a[j][e];
      }
    }
    scan_runs<V, P::kLanes>(A, B, eA, eB, at.lane);
    float start[V], tile_a[V], tile_b[V];
    if constexpr (NW > 1) {
      if (at.run == P::kRuns - 1) {
        Row<float, V>::store(&pair[buf][at.wave][0][at.ch], A);
        Row<float, V>::store(&pair[buf][at.wave][1][at.ch], B);
      }
      __syncthreads();  // the other buffer is written behind the next one
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        if (w == at.wave) {
#pragma unroll
          for (int e = 0; e < V; ++e) start[e] = carry[e];
        }
        float wa[V], wb[V];
        load_f32<V>(&pair[buf][w][0][at.ch], true, wa);
        load_f32<V>(&pair[buf][w][1][at.ch], true, wb);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if (SUM) {
            tile_b[e] = w == 0 ? wb[e] : fmaf(wa[e], tile_b[e], wb[e]);
            tile_a[e] = w == 0 ? wa[e] : tile_a[e] * wa[e];
          } else {
            carry[e] = fmaf(wa[e], carry[e], wb[e]);
          }
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        start[e] = carry[e];
        const int last = (P::kRuns - 1) * P::kLanes + at.lane % P::kLanes;
        const float wa = __shfl(A[e], last, 64), wb = __shfl(B[e], last, 64);
        tile_a[e] = wa;
        tile_b[e] = wb;
        if (!SUM) carry[e] = fmaf(wa, carry[e], wb);
      }
    }
    if (SUM) {  // in front of the tiles so far
#pragma unroll
      for (int e = 0; e < V; ++e) {
        carry[e] = fmaf(prod[e], tile_b[e], carry[e]);
        prod[e] *= tile_a[e];
      }
    }
    if constexpr (!SUM) {
      float h[V];
#pragma unroll
      for (int e = 0; e < V; ++e) h[e] = fmaf(eA[e], start[e], eB[e]);
      if (p.saved && chan && have > 0)
        Row<float, V>::store(p.saved + (bos / kRun + n + (t0 + at.token()) / kRun) * p.C + d, h);
      const __amdgpu_buffer_rsrc_t y = tile_of<E, P::kTokens>(p.y, bos + t0, t_end - t0, p.C);
#pragma unroll
      for (int j = 0; j < kRun; ++j) {
        float out[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          h[e] = fmaf(a[j][e], h[e], b[j][e]);
          out[e] = h[e];
          if constexpr (Z) {
            const float g = cz[j].get(e);
            out[e] = h[e] * (g * sigmoid_(g));
          }
        }
        Row<E, V>::store(y, first + j * step, out);
      }
    }
  }
  if (threadIdx.x < P::kLanes && chan) {
    if constexpr (SUM) {
      Row<float, V>::store(p.seg + (slot + s) * 2 * p.C + d, prod);
      Row<float, V>::store(p.seg + ((slot + s) * 2 + 1) * p.C + d, carry);
    } else if (p.h_final && t_begin + p.seg_len >= len) {
      Row<float, V>::store(p.h_final + static_cast<int64_t>(n) * p.C + d, carry);
    }
  }
}

// ---------------------------------------------------------------------------- backward

// Z: there is a gate.  SUM: the segments' (A, B) of K alone.
template <typename E, int V, int NW, bool Z, bool SUM>
__global__ __launch_bounds__(64 * NW) void glr_bwd_kernel(GlrParams p, int tiles) {
  using P = Place<V, NW>;
  const P at;
  const int tile = xcd_tile(blockIdx.x, tiles);
  if (tile >= tiles) return;
  const int n = blockIdx.y, s = blockIdx.z;
  int64_t bos, len;
  chunk::seq_range(p.seq, n, bos, len);
  const int64_t t_begin = s * p.seg_len, t_end = min(len, t_begin + p.seg_len);
  if (s > 0 && t_begin >= len) return;
  if (SUM && s == 0) return;  // nothing comes before the first
  const bool chan = tile * kGlrTile + at.ch < p.C;
  const int d = chan ? tile * kGlrTile + at.ch : 0;
  __shared__ alignas(16) float pair[2][NW][2][kGlrTile];

  float rate[V], carry[V], total[V], prod[V];
  load_f32<V>(p.lam + d, true, rate);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    rate[e] = rate_(rate[e], p.c);
    total[e] = 0.f;
    prod[e] = 1.f;
  }
  load_f32<V>(p.dh_final + static_cast<int64_t>(n) * p.C + d, p.dh_final != nullptr && !SUM, carry);
  const int64_t slot = bos / p.seg_len + n;
  if (!SUM) {
    const int last = len > 0 ? static_cast<int>((len - 1) / p.seg_len) : 0;
    for (int j = last; j > s; --j) {
      float a[V], b[V];
      load_f32<V>(p.seg + (slot + j) * 2 * p.C + d, true, a);
      load_f32<V>(p.seg + ((slot + j) * 2 + 1) * p.C + d, true, b);
#pragma unroll
      for (int e = 0; e < V; ++e) carry[e] = fmaf(a[e], carry[e], b[e]);
    }
  }

  const uint32_t step = static_cast<uint32_t>(p.C) * sizeof(E);
  const uint32_t first = chan ? static_cast<uint32_t>(at.token()) * step + static_cast<uint32_t>(d * sizeof(E)) : 0x7ffffff0u - kRun * step;
  // fp32 leaves no registers for a tile ahead
  constexpr bool kAhead = SUM || sizeof(E) == 2;
  Row<E, V> rx[kRun], rr[kRun], ri[kRun], rz[kRun], rd[kRun];
  Row<float, V> rh;
  auto fetch = [&](int64_t t0) {
    const __amdgpu_buffer_rsrc_t r = tile_of<E, P::kTokens>(p.r, bos + t0, t_end - t0, p.C), dy = tile_of<E, P::kTokens>(p.dy, bos + t0, t_end - t0, p.C);
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      rr[j].load(r, first + j * step);
      rd[j].load(dy, first + j * step);
    }
    if constexpr (Z) {
      const __amdgpu_buffer_rsrc_t z = tile_of<E, P::kTokens>(p.z, bos + t0, t_end - t0, p.C);
#pragma unroll
      for (int j = 0; j < kRun; ++j) rz[j].load(z, first + j * step);
    }
    if constexpr (!SUM) {
      const __amdgpu_buffer_rsrc_t x = tile_of<E, P::kTokens>(p.x, bos + t0, t_end - t0, p.C), gi = tile_of<E, P::kTokens>(p.i, bos + t0, t_end - t0, p.C);
#pragma unroll
      for (int j = 0; j < kRun; ++j) {
        rx[j].load(x, first + j * step);
        ri[j].load(gi, first + j * step);
      }
      rh.load(p.saved + (bos / kRun + n + min(t0 + at.token(), t_end - 1) / kRun) * p.C + d);
    }
  };
  // The pass for the sums goes from the segment's start to its end, as the next does not.
  const int64_t count = (t_end - t_begin + P::kTokens - 1) / P::kTokens;
  if (kAhead && count > 0) fetch(SUM ? t_begin : t_begin + (count - 1) * P::kTokens);
  int buf = 0;
  for (int64_t k = 0; k < count; ++k, buf ^= 1) {
    const int64_t t0 = t_begin + (SUM ? k : count - 1 - k) * P::kTokens;
    const int have = static_cast<int>(min(t_end - t0, static_cast<int64_t>(512))) - at.token();
    if (!kAhead) fetch(t0);
    Row<E, V> cx[kRun], cr[kRun], ci[kRun], cz[kRun], cd[kRun];
    float h[V];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      cx[j] = rx[j];
      cr[j] = rr[j];
      ci[j] = ri[j];
      if constexpr (Z) cz[j] = rz[j];
      cd[j] = rd[j];
    }
    if constexpr (!SUM) {
#pragma unroll
      for (int e = 0; e < V; ++e) h[e] = rh.get(e);
    }
    if (kAhead && k + 1 < count) fetch(SUM ? t0 + P::kTokens : t0 - P::kTokens);
    float a[kRun][V], before[kRun][V], ds[kRun][V];
    float A[V], B[V], eA[V], eB[V];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float la2 = rate[e] * sigmoid_(cr[j].get(e));
        const float decay = exp2_(la2);
        a[j][e] = decay;
        float g = cd[j].get(e);
        if constexpr (Z) {
          const float zz = cz[j].get(e);
          g *= zz * sigmoid_(zz);
        }
        ds[j][e] = g;
        if constexpr (!SUM) {
          before[j][e] = h[e];
          h[e] = fmaf(decay, h[e], root_(one_minus_square(la2, decay)) * sigmoid_(ci[j].get(e)) * cx[j].get(e));
        }
      }
    }
    if (t_end - t0 < P::kTokens) {  // behind the end a token changes nothing (ds is zero, as dy there)
#pragma unroll
      for (int j = 0; j < kRun; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) a[j][e] = j < have ? a[j][e] : 1.f;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      A[e] = 1.f;
      B[e] = 0.f;
#pragma unroll
      for (int j = kRun - 1; j >= 0; --j) {
        B[e] = a[j][e] * (ds[j][e] + B[e]);
        A[e] *= a[j][e];
      }
    }
    scan_runs_back<V, P::kLanes>(A, B, eA, eB, at.lane);
    float start[V], tile_a[V], tile_b[V];
    if constexpr (NW > 1) {
      if (at.run == 0) {
        Row<float, V>::store(&pair[buf][at.wave][0][at.ch], A);
        Row<float, V>::store(&pair[buf][at.wave][1][at.ch], B);
      }
      __syncthreads();
#pragma unroll
      for (int w = NW - 1; w >= 0; --w) {
        if (w == at.wave) {
#pragma unroll
          for (int e = 0; e < V; ++e) start[e] = carry[e];
        }
        float wa[V], wb[V];
        load_f32<V>(&pair[buf][w][0][at.ch], true, wa);
        load_f32<V>(&pair[buf][w][1][at.ch], true, wb);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if (SUM) {
            tile_b[e] = w == NW - 1 ? wb[e] : fmaf(wa[e], tile_b[e], wb[e]);
            tile_a[e] = w == NW - 1 ? wa[e] : tile_a[e] * wa[e];
          } else {
            carry[e] = fmaf(wa[e], carry[e], wb[e]);
          }
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        start[e] = carry[e];
        const float wa = __shfl(A[e], at.lane % P::kLanes, 64), wb = __shfl(B[e], at.lane % P::kLanes, 64);
        tile_a[e] = wa;
        tile_b[e] = wb;
        if (!SUM) carry[e] = fmaf(wa, carry[e], wb);
      }
    }
    if (SUM) {  // behind the tiles so far
#pragma unroll
      for (int e = 0; e < V; ++e) {
        carry[e] = fmaf(prod[e], tile_b[e], carry[e]);
        prod[e] *= tile_a[e];
      }
    }
    if constexpr (!SUM) {
      float K[V];
#pragma unroll
      for (int e = 0; e < V; ++e) K[e] = fmaf(eA[e], start[e], eB[e]);
      const __amdgpu_buffer_rsrc_t bx = tile_of<E, P::kTokens>(p.dx, bos + t0, t_end - t0, p.C), br = tile_of<E, P::kTokens>(p.dr, bos + t0, t_end - t0, p.C),
                                   bi = tile_of<E, P::kTokens>(p.di, bos + t0, t_end - t0, p.C);
#pragma unroll
      for (int j = kRun - 1; j >= 0; --j) {
        cr[j].forget();
        ci[j].forget();
        cx[j].forget();
        if constexpr (Z) {
          cz[j].forget();
          cd[j].forget();
        }
        float ox[V], orr[V], oi[V], oz[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float sr = sigmoid_(cr[j].get(e)), si = sigmoid_(ci[j].get(e)), xv = cx[j].get(e);
          const float la2 = rate[e] * sr, la = la2 * kLn2;
          const float decay = a[j][e], m = root_(one_minus_square(la2, decay));
          const float G = ds[j][e] + K[e];
          K[e] = decay * G;
          const float six = si * xv, hp = before[j][e];
          const float E1 = G * (decay * la * hp - decay * decay * (m > 0.f ? la * rcp_(m) : 0.f) * six);
          ox[e] = G * m * si;
          orr[e] = E1 * (1.f - sr);
          oi[e] = G * m * six * (1.f - si);
          if constexpr (Z) {
            const float zz = cz[j].get(e), sz = sigmoid_(zz);
            const float hn = fmaf(decay, hp, m * six);
            oz[e] = cd[j].get(e) * hn * sz * (1.f + zz * (1.f - sz));
          }
          total[e] += j < have ? E1 : 0.f;
        }
        Row<E, V>::store(bx, first + j * step, ox);
        Row<E, V>::store(br, first + j * step, orr);
        Row<E, V>::store(bi, first + j * step, oi);
        if (Z && p.dz) Row<E, V>::store(tile_of<E, P::kTokens>(p.dz, bos + t0, t_end - t0, p.C), first + j * step, oz);
      }
    }
  }
  if constexpr (SUM) {
    if (threadIdx.x < P::kLanes && chan) {
      Row<float, V>::store(p.seg + (slot + s) * 2 * p.C + d, prod);
      Row<float, V>::store(p.seg + ((slot + s) * 2 + 1) * p.C + d, carry);
    }
  } else {
    if (threadIdx.x < P::kLanes && chan && s == 0 && p.dh0) Row<float, V>::store(p.dh0 + static_cast<int64_t>(n) * p.C + d, carry);
    // the segment's sum of E, over the runs of a wave and then over the waves
#pragma unroll
    for (int e = 0; e < V; ++e)
#pragma unroll
      for (int off = P::kLanes; off < 64; off <<= 1) total[e] += __shfl_xor(total[e], off, 64);
    __syncthreads();
    if (at.run == 0) Row<float, V>::store(&pair[0][at.wave][0][at.ch], total);
    __syncthreads();
    if (threadIdx.x < P::kLanes && chan) {
      float sum[V];
#pragma unroll
      for (int e = 0; e < V; ++e) sum[e] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += pair[0][w][0][at.ch + e];
      Row<float, V>::store(p.part_lam + (slot + s) * p.C + d, sum);
    }
  }
}

// dlam from the segments' sums, 64 channels a workgroup: each of four waves adds every
// fourth sequence's in order, then the four are added.
__global__ __launch_bounds__(256) void glr_lam_kernel(GlrParams p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, d = blockIdx.x * 64 + lane;
  __shared__ float part[4][64];
  float sum = 0.f;
  if (d < p.C) {
    for (int n = wave; n < p.N; n += 4) {
      int64_t bos, len;
      chunk::seq_range(p.seq, n, bos, len);
      const int64_t slot = bos / p.seg_len + n, count = (len + p.seg_len - 1) / p.seg_len;
      for (int64_t j = 0; j < count; ++j) sum += p.part_lam[(slot + j) * p.C + d];
    }
  }
  part[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && d < p.C) {
    sum = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
    float sig;
    const float soft = softplus_(p.lam[d], sig);
    // both are exp(lam) where that underflows
    p.dlam[d] = soft > 0.f ? sum * (sig / soft) : sum;
  }
}

// ---------------------------------------------------------------------------- one token

template <typename E, int V>
__global__ __launch_bounds__(256) void glr_step_kernel(GlrParams p) {
  const int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, at = v * V;
  if (at >= p.rows * p.C) return;
  const int d = static_cast<int>(at % p.C);
  Row<E, V> rx, rr, ri, rz;
  rx.load(static_cast<const E*>(p.x) + at);
  rr.load(static_cast<const E*>(p.r) + at);
  ri.load(static_cast<const E*>(p.i) + at);
  if (p.z) rz.load(static_cast<const E*>(p.z) + at);
  float h[V], lam[V], out[V];
  load_f32<V>(p.h_final + at, true, h);
  load_f32<V>(p.lam + d, true, lam);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float la2 = rate_(lam[e], p.c) * sigmoid_(rr.get(e)), decay = exp2_(la2);
    h[e] = fmaf(decay, h[e], root_(one_minus_square(la2, decay)) * sigmoid_(ri.get(e)) * rx.get(e));
    out[e] = h[e];
    if (p.z) {
      const float g = rz.get(e);
      out[e] = h[e] * (g * sigmoid_(g));
    }
  }
  Row<float, V>::store(p.h_final + at, h);
  Row<E, V>::store(static_cast<E*>(p.y) + at, out);
}

dim3 grid_of(const GlrParams& p, int tiles) {
  return dim3(static_cast<unsigned>((tiles + 7) / 8 * 8), static_cast<unsigned>(p.N), static_cast<unsigned>(p.segs));
}

template <typename E, int NW, bool Z>
void fwd(const GlrParams& p, hipStream_t s) {
  constexpr int V = glr_vec(false, sizeof(E) == 2);
  const int tiles = glr_tiles(p.C);
  if (p.segs > 1) hipLaunchKernelGGL((glr_fwd_kernel<E, V, NW, false, true>), grid_of(p, tiles), dim3(64 * NW), 0, s, p, tiles);
  hipLaunchKernelGGL((glr_fwd_kernel<E, V, NW, Z, false>), grid_of(p, tiles), dim3(64 * NW), 0, s, p, tiles);
}

template <typename E, int NW, bool Z>
void bwd(const GlrParams& p, hipStream_t s) {
  constexpr int V = glr_vec(true, sizeof(E) == 2);
  const int tiles = glr_tiles(p.C);
  if (p.segs > 1) hipLaunchKernelGGL((glr_bwd_kernel<E, V, NW, Z, true>), grid_of(p, tiles), dim3(64 * NW), 0, s, p, tiles);
  if (p.N > 0) hipLaunchKernelGGL((glr_bwd_kernel<E, V, NW, Z, false>), grid_of(p, tiles), dim3(64 * NW), 0, s, p, tiles);
  hipLaunchKernelGGL(glr_lam_kernel, dim3(static_cast<unsigned>((p.C + 63) / 64)), dim3(256), 0, s, p);
}

template <typename E, int NW, bool BWD>
hipError_t launch(const GlrParams& p, hipStream_t s) {
  if constexpr (BWD)
    p.z ? bwd<E, NW, true>(p, s) : bwd<E, NW, false>(p, s);
  else
    p.z ? fwd<E, NW, true>(p, s) : fwd<E, NW, false>(p, s);
  return hipGetLastError();
}

template <typename E, bool BWD>
hipError_t launch_waves(const GlrParams& p, hipStream_t s) {
  switch (p.waves) {
    case 1: return launch<E, 1, BWD>(p, s);
    case 4: return launch<E, 4, BWD>(p, s);
    default: return launch<E, 8, BWD>(p, s);
  }
}

}  // namespace

hipError_t launch_glr_fwd(const GlrParams& p, bool bf16, hipStream_t s) {
  return bf16 ? launch_waves<uint16_t, false>(p, s) : launch_waves<float, false>(p, s);
}

hipError_t launch_glr_bwd(const GlrParams& p, bool bf16, hipStream_t s) {
  return bf16 ? launch_waves<uint16_t, true>(p, s) : launch_waves<float, true>(p, s);
}

hipError_t launch_glr_step(const GlrParams& p, bool bf16, hipStream_t s) {
  const int64_t values = p.rows * p.C;
  const int V = bf16 ? 8 : 4;
  const unsigned blocks = static_cast<unsigned>((values / V + 255) / 256);
  if (bf16)
    hipLaunchKernelGGL((glr_step_kernel<uint16_t, 8>), dim3(blocks), dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((glr_step_kernel<float, 4>), dim3(blocks), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace gdn
