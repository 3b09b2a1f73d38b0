// Device parts shared by the selective scan's forward and backward kernels: the
// channel tile of a workgroup, the staging of a tile of tokens in LDS, and the lane
// reductions.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_layer.h"
#include "gdn_layer_device.h"

// The instance for a state count (8, 16, 32, 64) and an io dtype.
#define GDN_SCAN_DISPATCH(fn)                                                     \
  switch (N) {                                                                    \
    case 8: return bf16 ? fn<uint16_t, 8>(p, s) : fn<float, 8>(p, s);             \
    case 16: return bf16 ? fn<uint16_t, 16>(p, s) : fn<float, 16>(p, s);          \
    case 32: return bf16 ? fn<uint16_t, 32>(p, s) : fn<float, 32>(p, s);          \
    default: return bf16 ? fn<uint16_t, 64>(p, s) : fn<float, 64>(p, s);          \
  }

namespace gdn {
namespace scan {

using namespace layer;

// Wave priorities in the scan kernels (s_setprio): decays and writes before the chain
// through them, that before staging and stores.  Without them the eldest workgroup of a
// SIMD goes first all the time, all are in the same part more often, and the youngest ends
// by itself: with equal work, two workgroups a CU took 85 and 104 us.

constexpr int kTile = 16;     // tokens staged at a time
constexpr int kYStride = 80;  // row stride of output tiles: the four token rows a wave writes fall in other banks

// A workgroup's channels d0 .. d0 + count - 1, all of group g.
struct ChannelTile {
  int g, tile, d0, count;  // tile: its number in the group
  __device__ __forceinline__ ChannelTile(const ScanParams& p, int block) {
    const int per = p.D / p.G, tiles = (per + kScanTile - 1) / kScanTile;
    g = block / tiles;
    tile = block - g * tiles;
    const int at = tile * kScanTile;
    d0 = g * per + at;
    count = min(kScanTile, per - at);
  }
};

// Slot of the state kept before token t (a multiple of kScanBlock) of sequence n.
__device__ __forceinline__ int64_t saved_slot(int64_t bos, int n, int64_t t) {
  return bos / kScanBlock + n + t / kScanBlock;
}

// Slot of segment `seg` of sequence n in the buffers of segments; its slots and those of
// the next sequence (the slots behind its last segment are at most two).
__device__ __forceinline__ int64_t part_slot(const ScanParams& p, int64_t bos, int n, int seg) {
  return bos / p.seg_len + n + seg;
}

template <int S>
__device__ __forceinline__ void load_states(const float* p, bool ok, float (&f)[S]) {
#pragma unroll
  for (int s = 0; s < S; ++s) f[s] = 0.f;
  if (!ok) return;
  if constexpr (S == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    f[0] = v.x; f[1] = v.y;
  } else {
#pragma unroll
    for (int s = 0; s < S; s += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + s);
      f[s] = v.x; f[s + 1] = v.y; f[s + 2] = v.z; f[s + 3] = v.w;
    }
  }
}
template <int S>
__device__ __forceinline__ void read_states(const float* p, float (&f)[S]) {
  load_states<S>(p, true, f);
}
template <int S>
__device__ __forceinline__ void store_states(float* p, const float (&f)[S]) {
  if constexpr (S == 2) {
    *reinterpret_cast<float2*>(p) = float2{f[0], f[1]};
  } else {
#pragma unroll
    for (int s = 0; s < S; s += 4) *reinterpret_cast<float4*>(p + s) = float4{f[s], f[s + 1], f[s + 2], f[s + 3]};
  }
}

typedef uint32_t u32pair_t __attribute__((ext_vector_type(2)));
// a: lanes 0-31 of a, then lanes 0-31 of b; b: lanes 32-63 of a, then of b.
__device__ __forceinline__ void swap32(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
// The same between the odd row of 16 lanes of a and the even one of b, in each half.
__device__ __forceinline__ void swap16(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
// Lane 16 q + c gets x_q summed over the four rows of lanes (0..3) at c.
__device__ __forceinline__ float reduce_rows4(float x0, float x1, float x2, float x3) {
  swap32(x0, x2);
  swap32(x1, x3);
  float a = x0 + x2, b = x1 + x3;
  swap16(a, b);
  return a + b;
}

// A tile of TT tokens in LDS: (delta, delta u) of every channel, B and C rows in
// fp32, PAD more values a row.  Tokens behind the end hold zeros, which leave the state as it
// is.
template <int N, int TT, int PAD = 0>
struct Stage {
  float2 dd[TT][kScanTile];
  float B[TT][N + PAD];
  float C[TT][N + PAD];
};

// dt_bias and D of the tile's channels (zero where there is none), in LDS: registers
// are scarce across a tile.  Filled by one workgroup barrier before its use.
struct ChannelParams {
  float bias[kScanTile], skip[kScanTile];
  __device__ __forceinline__ void fill(const ScanParams& p, const ChannelTile& ct) {
    const int c = threadIdx.x;
    if (c < kScanTile) {
      bias[c] = p.dt_bias && c < ct.count ? p.dt_bias[ct.d0 + c] : 0.f;
      skip[c] = p.Dskip && c < ct.count ? p.Dskip[ct.d0 + c] : 0.f;
    }
  }
};

// A thread's share of a tile of TT tokens: EL channels of one token (row, col), and
// a piece of that token's B and C.
template <typename E, int N, int TT>
struct Loader {
  static constexpr int EL = TT / 4;            // 64 channels over 256 / TT threads
  static constexpr int kPer = 256 / TT;        // threads of a token
  static constexpr int P = N > kPer ? N / kPer : 1;
  const ScanParams& p;
  int64_t bos;
  int g, d, row, col, piece;
  bool live, has_z;
  Raw<E, EL> u, dt, z;
  E b[P], c[P];

  __device__ __forceinline__ Loader(const ScanParams& p_, const ChannelTile& ct, int64_t bos_, bool has_z_)
      : p(p_), bos(bos_), g(ct.g), has_z(has_z_) {
    row = threadIdx.x / kPer;
    piece = threadIdx.x % kPer;
    col = piece * EL;
    live = col < ct.count;
    d = ct.d0 + (live ? col : 0);
  }
  __device__ __forceinline__ int64_t token(int64_t t0, int64_t end) const { return bos + min(t0 + row, end - 1); }
  __device__ __forceinline__ void fetch(int64_t t0, int64_t end) {
    const int64_t t = token(t0, end);
    u.load(static_cast<const E*>(p.u) + t * p.D + d);
    dt.load(static_cast<const E*>(p.dt) + t * p.D + d);
    if (has_z) z.load(static_cast<const E*>(p.z) + t * p.D + d);
    const int64_t bc = (t * p.G + g) * N + (piece * P < N ? piece * P : 0);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      b[i] = static_cast<const E*>(p.Bm)[bc + i];
      c[i] = static_cast<const E*>(p.Cm)[bc + i];
    }
  }
  // `delta` and its derivative `sig` by dt of this thread's channels (zero behind the end)
  template <int PAD>
  __device__ __forceinline__ void put(Stage<N, TT, PAD>& st, const ChannelParams& cp, int64_t t0, int64_t end,
                                      float (&delta)[EL], float (&sig)[EL]) const {
    const bool ok = t0 + row < end, both = ok && live;
    float2 v[EL];
#pragma unroll
    for (int e = 0; e < EL; ++e) {
      delta[e] = dt.get(e) + cp.bias[col + e];
      sig[e] = 1.f;
    }
    if (p.softplus) {
#pragma unroll
      for (int e = 0; e < EL; ++e) delta[e] = softplus_(delta[e], sig[e]);
    }
#pragma unroll
    for (int e = 0; e < EL; ++e) {
      delta[e] = both ? delta[e] : 0.f;
      const float du = delta[e] * u.get(e);
      v[e] = float2{delta[e], both ? du : 0.f};
    }
#pragma unroll
    for (int e = 0; e < EL; e += 2)
      *reinterpret_cast<float4*>(&st.dd[row][col + e]) = float4{v[e].x, v[e].y, v[e + 1].x, v[e + 1].y};
    if (piece * P < N) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        st.B[row][piece * P + i] = ok ? IoT<E>::ld(&b[i]) : 0.f;
        st.C[row][piece * P + i] = ok ? IoT<E>::ld(&c[i]) : 0.f;
      }
    }
  }
};

}  // namespace scan
}  // namespace gdn
