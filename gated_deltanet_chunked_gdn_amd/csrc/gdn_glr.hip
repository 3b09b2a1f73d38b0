// The gated linear recurrence on gfx950: per sequence and channel
//
//   la = -c softplus(lam) sigmoid(r_t);  a = exp(la);  m = sqrt(1 - a^2)
//   h <- a h + m sigmoid(i_t) x_t;  y_t = h  or  h silu(z_t)
//
// A linear recurrence composes: a run of tokens takes h to A h + B, with A the product of
// its decays and B its end from zero.  A workgroup holds a segment of 64 channels (rows of
// 128 or 256 bytes; at 64 bytes the same loads took a third longer) in registers, runs of eight tokens a
// thread: it forms every run's (A, B), composes them by lane shifts inside a wave and through
// LDS between waves, learns the state in front of the segment, and goes through the runs once
// more.  So all is read once, and the segments of a sequence work at the same time.
//
// The state in front comes from the other segments.  Each gives out its (A, B) as soon as it
// has them.  Some segments are a group: a segment composes those of its group before it,
// all loaded at once, onto the group's start, and the group's last one gives out the next
// group's.  The order of every composition is fixed, whoever comes first, so results are
// bit-identical from call to call.  The words that pass carry a mark beside the value and are
// single 64-bit stores and loads of device scope, so a value cannot be taken before it is
// there, and nothing else need be ordered.  Segments are counted off as workgroups start,
// earlier ones of a sequence first, so a workgroup waits only for others that already run and
// wait for none behind it: the first that has not ended never waits.  The wait is bounded all
// the same (a state of NaN follows, for calls that share a workspace against the rules).
//
// Backward.  With K_t = dL/dh_t through the later tokens and ds_t = dL/dh_t through y_t,
//   G_t = ds_t + K_t;  K_{t-1} = a_t G_t
// which is the same recurrence from the end; states come from those that the forward keeps
// every eight tokens (1/16 of what it reads, and exact in fp32).  With la times its own
// gradient no quotient grows without bound (m ~ sqrt(-2 la) where la is small):
//   E = G (a la h_{t-1} - a^2 (la / m) sigmoid(i) x)
//   dr = E (1 - sigmoid(r));  dlam = sum_t E sigmoid(lam) / softplus(lam)
//   dx = G m sigmoid(i);  di = G m x sigmoid(i) (1 - sigmoid(i));  dz = dy h silu'(z)
//
// HBM-bound.  Forward of 65536 x 1024 with a gate, bf16: 170 us, 3.95 TB/s of the 671 MB it reads
// and writes (a large copy: 5.1); 4 x 4096 x 2048: 98 us.  Backward of the latter: 172 to 177 us, 3.5 TB/s of
// its 621 MB, and 5 each for the clearing of the words and for dlam.  With two passes over the
// inputs instead of words that pass on, 252 us and, training, 332 against 263.
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
    else if constexpr (kWords == 2)
      w = __builtin_bit_cast(vec_t, __builtin_amdgcn_raw_buffer_load_b64(r, byte, 0, 0));
    else
      w = __builtin_bit_cast(vec_t, __builtin_amdgcn_raw_buffer_load_b128(r, byte, 0, 0));
  }
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t byte, const float* f) {
    vec_t v;
#pragma unroll
    for (int i = 0; i < kWords; ++i) v[i] = sizeof(E) == 2 ? pack_bf16x2(f[2 * i], f[2 * i + 1]) : __float_as_uint(f[i]);
    if constexpr (kWords == 1)
      __builtin_amdgcn_raw_buffer_store_b32(v[0], r, byte, 0, 0);
    else if constexpr (kWords == 2)
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(chunk::u32x2v_t, v), r, byte, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(chunk::u32x4v_t, v), r, byte, 0, 0);
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

// A tile's rows of one tensor, as a resource that ends with the segment, which is `left` rows
// off: at most 2^29 bytes (128 rows of 2^20 values).
template <typename E, int ROWS>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_of(const void* base, int64_t row, int64_t left, int C) {
  static_assert(ROWS <= 128, "2^29 bytes");
  const int64_t rows = min(left, static_cast<int64_t>(ROWS));
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(static_cast<const E*>(base) + row * C), 0,
                                           static_cast<int>(static_cast<uint32_t>(rows) * C * sizeof(E)), 0x00020000);
}

// What a workgroup works on, and where its threads stand in it.
template <int V>
struct Place {
  static constexpr int kLanes = kGlrTile / V;                  // lanes of a row
  static constexpr int kRuns = 64 / kLanes;                    // runs of a wave
  static constexpr int kTokens = kRuns * kRun * kGlrWaves;     // of a segment
  int lane, wave, run, ch;  // ch: first channel in the tile's 64
  int n, seg, segs;         // sequence, segment (from its start), its segments
  int64_t bos, len, t0;     // t0: the segment's first token
  int64_t slot;
  int tile;
  bool live;
  __device__ __forceinline__ int token() const { return (wave * kRuns + run) * kRun; }
  // `index` counts workgroups; `back`: later segments of a sequence come first
  __device__ __forceinline__ Place(const GlrParams& p, int64_t index, int tiles, bool back) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    run = lane / kLanes;
    ch = (lane % kLanes) * V;
    slot = glr_slot(index, tiles, p.slots, back);
    tile = static_cast<int>(index % tiles);
    // the sequence whose slots hold this one: the last that starts at or before it
    int lo = 0, hi = p.N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start(p, mid) <= slot)
        lo = mid;
      else
        hi = mid;
    }
    n = lo;
    seg = static_cast<int>(slot - start(p, n));
    chunk::seq_range(p.seq, n, bos, len);
    segs = static_cast<int>(max((len + kTokens - 1) / kTokens, static_cast<int64_t>(1)));
    t0 = static_cast<int64_t>(seg) * kTokens;
    live = slot >= 0 && seg < segs;  // an empty sequence has one segment, of no tokens
  }
  // A sequence's first slot.  Dense ones have the slots that their segments need and no more.
  static __device__ __forceinline__ int64_t start(const GlrParams& p, int n) {
    return p.seq.cu ? p.seq.cu[n] / kTokens + n : static_cast<int64_t>(n) * (p.slots / p.N);
  }
};

// The workgroup's number: in the order in which they start where they wait for each other.
__device__ __forceinline__ int64_t number(const GlrParams& p) {
  if (!p.chained) return blockIdx.x;
  __shared__ uint32_t mine;
  if (threadIdx.x == 0)
    mine = __hip_atomic_fetch_add(reinterpret_cast<uint32_t*>(p.chain), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(mine));
}

// Words that workgroups pass to each other; zero: not there yet.  A state stands beside a one;
// of a segment's (A, B), A is positive or zero (or NaN), so its sign is the mark.
// A word is one atomic access of 64 bits, the widest that there are, of device scope: past the
// caches of an XCD (sc1), neither merged nor moved.  Word e of lane l of a tile's row of channels
// stands at e kLanes + l, so that an access of the lanes is one piece of memory (channels in
// order: 178 us for 172, 65536 x 1024).
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));  // value, mark
template <int V, int LANES>
__device__ __forceinline__ void give_(uint64_t* to, uint32_t off, const u32x2_t* w) {
  uint64_t* const p = reinterpret_cast<uint64_t*>(reinterpret_cast<char*>(to) + off);
#pragma unroll
  for (int e = 0; e < V; ++e) __hip_atomic_store(p + e * LANES, __builtin_bit_cast(uint64_t, w[e]), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Waits until all words of all lanes of the wave are there: V at each place, `off` bytes from
// `from`; lanes that want none of a place say so.
template <int V, int LANES, int COUNT>
__device__ __forceinline__ void take_(const uint64_t* from, const uint32_t* off, const bool* want, u32x2_t (*w)[V]) {
  bool missing[COUNT];
#pragma unroll
  for (int i = 0; i < COUNT; ++i) missing[i] = want[i];
  for (int tries = 0;; ++tries) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
      if (missing[i]) {
#pragma unroll
        for (int e = 0; e < V; ++e)
          w[i][e] = __builtin_bit_cast(u32x2_t, __hip_atomic_load(reinterpret_cast<const uint64_t*>(reinterpret_cast<const char*>(from) + off[i]) + e * LANES,
                                                                  __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
      }
    bool there = true;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      if (missing[i]) {
        missing[i] = false;
#pragma unroll
        for (int e = 0; e < V; ++e) missing[i] |= w[i][e][1] == 0;
      }
      there &= !missing[i];
    }
    if (__all(there)) return;
    if (tries >= 1 << 20) {  // about a second: whoever should give it shares its workspace with another call
#pragma unroll
      for (int i = 0; i < COUNT; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) w[i][e] = u32x2_t{0x7fc00000u, 0x7fc00000u};
      return;
    }
    __builtin_amdgcn_s_sleep(2);
  }
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

// (A, B) of a wave's runs by wave, in LDS; and of the segments before, by wave.
struct Shared {
  alignas(16) float wave[kGlrWaves][2][kGlrTile];
  alignas(16) float before[kGlrWaves][2][kGlrTile];
  alignas(16) float start[kGlrTile];
};

// The state in front of the segment, for this thread's channels: `carry` holds the sequence's
// own (the first group's start), `a`, `b` the segment's (A, B).  `place` counts segments in the
// direction of the walk.  Called by the whole workgroup.
template <int V>
__device__ __forceinline__ void arrive(const GlrParams& p, Shared& sh, const Place<V>& at, int place, int64_t first_slot, int dir,
                                       bool chan, const float* a, const float* b, float* carry) {
  using P = Place<V>;
  const int group = place / kGlrGroup, index = place % kGlrGroup;
  const int64_t group_slot = at.bos / (P::kTokens * kGlrGroup) + at.n;
  const bool lead = threadIdx.x < P::kLanes && chan;
  // of channels behind the last: words that are given all the same
  const uint32_t lane_off = chan ? static_cast<uint32_t>(at.tile * kGlrTile + at.ch / V) * 8 : 0;
  if (place + 1 < at.segs && index + 1 < kGlrGroup && lead) {
    u32x2_t w[V];
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = u32x2_t{__float_as_uint(b[e]), __float_as_uint(a[e]) | 0x80000000u};
    give_<V, P::kLanes>(p.whole + (first_slot + dir * place) * p.words, lane_off, w);
  }
  if (place == 0) return;
  // The segments of the group before this one, a few consecutive ones for every run of the
  // workgroup's lanes, all loaded at once.
  constexpr int kPlaces = P::kRuns * kGlrWaves, kEach = kGlrGroup > kPlaces ? kGlrGroup / kPlaces : 1;
  float ca[V], cb[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    ca[e] = 1.f;
    cb[e] = 0.f;
  }
  {
    u32x2_t w[kEach][V];
    uint32_t off[kEach];
    bool want[kEach];
    // the lowest slot of them: walked backwards, the nearest
    const int64_t lowest = first_slot + dir * (dir > 0 ? group * kGlrGroup : place - 1);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int k = (at.wave * P::kRuns + at.run) * kEach + i;
      want[i] = k < index;
      off[i] = lane_off + static_cast<uint32_t>(want[i] ? (dir > 0 ? k : index - 1 - k) : 0) * p.words * 8;
    }
    take_<V, P::kLanes, kEach>(p.whole + lowest * p.words, off, want, w);
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (want[i]) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float sa = __uint_as_float(w[i][e][1] & 0x7fffffffu);
          cb[e] = fmaf(sa, cb[e], __uint_as_float(w[i][e][0]));
          ca[e] *= sa;
        }
      }
  }
  // the wave's, in order of its runs
#pragma unroll
  for (int off = P::kLanes; off < 64; off <<= 1) {
    const bool later = at.lane & off;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float oa = __shfl_xor(ca[e], off, 64), ob = __shfl_xor(cb[e], off, 64);
      cb[e] = later ? fmaf(ca[e], ob, cb[e]) : fmaf(oa, cb[e], ob);
      ca[e] *= oa;
    }
  }
  if (at.run == 0) {
    Row<float, V>::store(&sh.before[at.wave][0][at.ch], ca);
    Row<float, V>::store(&sh.before[at.wave][1][at.ch], cb);
  }
  if (group > 0 && at.wave == 0) {
    u32x2_t w[1][V];
    const bool want[1] = {at.run == 0};
    take_<V, P::kLanes, 1>(p.end + (group_slot + group - 1) * p.words, &lane_off, want, w);
    if (at.run == 0) {
      float f[V];
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = __uint_as_float(w[0][e][0]);
      Row<float, V>::store(&sh.start[at.ch], f);
    }
  }
  __syncthreads();
  if (group > 0) load_f32<V>(&sh.start[at.ch], true, carry);
#pragma unroll
  for (int w = 0; w < kGlrWaves; ++w) {
    float wa[V], wb[V];
    load_f32<V>(&sh.before[w][0][at.ch], true, wa);
    load_f32<V>(&sh.before[w][1][at.ch], true, wb);
#pragma unroll
    for (int e = 0; e < V; ++e) carry[e] = fmaf(wa[e], carry[e], wb[e]);
  }
  if (index + 1 == kGlrGroup && place + 1 < at.segs && lead) {
    u32x2_t w[V];
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = u32x2_t{__float_as_uint(fmaf(a[e], carry[e], b[e])), 1u};
    give_<V, P::kLanes>(p.end + (group_slot + group) * p.words, lane_off, w);
  }
}

// ---------------------------------------------------------------------------- forward

// Z: there is a gate.
template <typename E, int V, bool Z>
__global__ __launch_bounds__(64 * kGlrWaves, sizeof(E) == 2 ? 3 : 2) void glr_fwd_kernel(GlrParams p, int tiles) {
  using P = Place<V>;
  const P at(p, number(p), tiles, false);
  if (!at.live) return;
  const bool chan = at.tile * kGlrTile + at.ch < p.C;  // whole vectors: C is a multiple of 8
  const int d = chan ? at.tile * kGlrTile + at.ch : 0;
  const int64_t row = at.bos + at.t0, left = at.len - at.t0;
  const int have = static_cast<int>(min(left, static_cast<int64_t>(P::kTokens))) - at.token();  // tokens of the run and behind it
  // offset of this thread's run; of channels behind the last, behind every tile's end
  const uint32_t step = static_cast<uint32_t>(p.C) * sizeof(E);
  const uint32_t first = chan ? static_cast<uint32_t>(at.token()) * step + static_cast<uint32_t>(d * sizeof(E)) : 0x7ffffff0u - kRun * step;
  __shared__ Shared sh;

  Row<E, V> rx[kRun], rr[kRun], ri[kRun], rz[kRun];
  {
    const __amdgpu_buffer_rsrc_t x = tile_of<E, P::kTokens>(p.x, row, left, p.C), r = tile_of<E, P::kTokens>(p.r, row, left, p.C),
                                 gi = tile_of<E, P::kTokens>(p.i, row, left, p.C);
#pragma unroll
    for (int j = 0; j < kRun; ++j) rr[j].load(r, first + j * step);
#pragma unroll
    for (int j = 0; j < kRun; ++j) ri[j].load(gi, first + j * step);
#pragma unroll
    for (int j = 0; j < kRun; ++j) rx[j].load(x, first + j * step);
    if constexpr (Z) {
      const __amdgpu_buffer_rsrc_t z = tile_of<E, P::kTokens>(p.z, row, left, p.C);
#pragma unroll
      for (int j = 0; j < kRun; ++j) rz[j].load(z, first + j * step);
    }
  }
  float rate[V], carry[V];
  load_f32<V>(p.lam + d, true, rate);
#pragma unroll
  for (int e = 0; e < V; ++e) rate[e] = rate_(rate[e], p.c);
  load_f32<V>(p.h0 + static_cast<int64_t>(at.n) * p.C + d, p.h0 != nullptr, carry);

  float a[kRun][V], b[kRun][V];
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float la2 = rate[e] * sigmoid_(rr[j].get(e));
      const float decay = exp2_(la2);
      a[j][e] = decay;
      b[j][e] = root_(one_minus_square(la2, decay)) * sigmoid_(ri[j].get(e)) * rx[j].get(e);
    }
  }
  if (left < P::kTokens) {  // behind the end a token changes nothing (b is zero, as x there)
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
  if (at.run == P::kRuns - 1) {
    Row<float, V>::store(&sh.wave[at.wave][0][at.ch], A);
    Row<float, V>::store(&sh.wave[at.wave][1][at.ch], B);
  }
  __syncthreads();
  float fa[V], fb[V];  // the segment's
#pragma unroll
  for (int w = 0; w < kGlrWaves; ++w) {
    float wa[V], wb[V];
    load_f32<V>(&sh.wave[w][0][at.ch], true, wa);
    load_f32<V>(&sh.wave[w][1][at.ch], true, wb);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (w == at.wave) {  // the runs before this one, in the segment
        const float sa = w ? fa[e] : 1.f, sb = w ? fb[e] : 0.f;
        eB[e] = fmaf(eA[e], sb, eB[e]);
        eA[e] *= sa;
      }
      fb[e] = w ? fmaf(wa[e], fb[e], wb[e]) : wb[e];
      fa[e] = w ? fa[e] * wa[e] : wa[e];
    }
  }
  arrive<V>(p, sh, at, at.seg, P::start(p, at.n), 1, chan, fa, fb, carry);

  float h[V];
#pragma unroll
  for (int e = 0; e < V; ++e) h[e] = fmaf(eA[e], carry[e], eB[e]);
  if (p.saved && chan && have > 0)
    Row<float, V>::store(p.saved + (at.bos / kRun + at.n + (at.t0 + at.token()) / kRun) * p.C + d, h);
  const __amdgpu_buffer_rsrc_t y = tile_of<E, P::kTokens>(p.y, row, left, p.C);
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
    float out[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      h[e] = fmaf(a[j][e], h[e], b[j][e]);
      out[e] = h[e];
      if constexpr (Z) {
        const float g = rz[j].get(e);
        out[e] = h[e] * (g * sigmoid_(g));
      }
    }
    Row<E, V>::store(y, first + j * step, out);
  }
  if (threadIdx.x < P::kLanes && chan && p.h_final && at.seg + 1 == at.segs) {
    float last[V];
#pragma unroll
    for (int e = 0; e < V; ++e) last[e] = fmaf(fa[e], carry[e], fb[e]);
    Row<float, V>::store(p.h_final + static_cast<int64_t>(at.n) * p.C + d, last);
  }
}

// ---------------------------------------------------------------------------- backward

// Without a gate four waves a SIMD: 4 x 4096 x 2048 both ways 220 us, with three (two registers more) 225.
template <typename E, int V, bool Z>
__global__ __launch_bounds__(64 * kGlrWaves, sizeof(E) == 2 ? (Z ? 3 : 4) : 2) void glr_bwd_kernel(GlrParams p, int tiles) {
  using P = Place<V>;
  const P at(p, number(p), tiles, true);
  if (at.slot < 0) return;
  const bool chan = at.tile * kGlrTile + at.ch < p.C;
  if (!at.live) {  // a slot between two sequences'
    if (threadIdx.x < P::kLanes && chan) {
      const float none[V] = {};
      Row<float, V>::store(p.part_lam + at.slot * p.C + at.tile * kGlrTile + at.ch, none);
    }
    return;
  }
  const int d = chan ? at.tile * kGlrTile + at.ch : 0;
  const int64_t row = at.bos + at.t0, left = at.len - at.t0;
  const int have = static_cast<int>(min(left, static_cast<int64_t>(P::kTokens))) - at.token();
  const uint32_t step = static_cast<uint32_t>(p.C) * sizeof(E);
  const uint32_t first = chan ? static_cast<uint32_t>(at.token()) * step + static_cast<uint32_t>(d * sizeof(E)) : 0x7ffffff0u - kRun * step;
  __shared__ Shared sh;

  Row<E, V> rx[kRun], rr[kRun], ri[kRun], rz[kRun], rd[kRun];
  float h[V];
  {
    const __amdgpu_buffer_rsrc_t r = tile_of<E, P::kTokens>(p.r, row, left, p.C), dy = tile_of<E, P::kTokens>(p.dy, row, left, p.C),
                                 x = tile_of<E, P::kTokens>(p.x, row, left, p.C), gi = tile_of<E, P::kTokens>(p.i, row, left, p.C);
#pragma unroll
    for (int j = 0; j < kRun; ++j) rr[j].load(r, first + j * step);
#pragma unroll
    for (int j = 0; j < kRun; ++j) rd[j].load(dy, first + j * step);
    if constexpr (Z) {
      const __amdgpu_buffer_rsrc_t z = tile_of<E, P::kTokens>(p.z, row, left, p.C);
#pragma unroll
      for (int j = 0; j < kRun; ++j) rz[j].load(z, first + j * step);
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j) ri[j].load(gi, first + j * step);
#pragma unroll
    for (int j = 0; j < kRun; ++j) rx[j].load(x, first + j * step);
    load_f32<V>(p.saved + (at.bos / kRun + at.n + (at.t0 + at.token()) / kRun) * p.C + d, have > 0, h);
  }
  float rate[V], carry[V];
  load_f32<V>(p.lam + d, true, rate);
#pragma unroll
  for (int e = 0; e < V; ++e) rate[e] = rate_(rate[e], p.c);
  load_f32<V>(p.dh_final + static_cast<int64_t>(at.n) * p.C + d, p.dh_final != nullptr, carry);

  float a[kRun][V], ds[kRun][V];
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      a[j][e] = exp2_(rate[e] * sigmoid_(rr[j].get(e)));
      float g = rd[j].get(e);
      if constexpr (Z) {
        const float zz = rz[j].get(e);
        g *= zz * sigmoid_(zz);
      }
      ds[j][e] = g;
    }
  }
  if (left < P::kTokens) {  // behind the end a token changes nothing (ds is zero, as dy there)
#pragma unroll
    for (int j = 0; j < kRun; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) a[j][e] = j < have ? a[j][e] : 1.f;
  }
  float A[V], B[V], eA[V], eB[V];
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
  if (at.run == 0) {
    Row<float, V>::store(&sh.wave[at.wave][0][at.ch], A);
    Row<float, V>::store(&sh.wave[at.wave][1][at.ch], B);
  }
  __syncthreads();
  float fa[V], fb[V];
#pragma unroll
  for (int w = kGlrWaves - 1; w >= 0; --w) {
    const bool none = w == kGlrWaves - 1;
    float wa[V], wb[V];
    load_f32<V>(&sh.wave[w][0][at.ch], true, wa);
    load_f32<V>(&sh.wave[w][1][at.ch], true, wb);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (w == at.wave) {  // the runs behind this one, in the segment
        const float sa = none ? 1.f : fa[e], sb = none ? 0.f : fb[e];
        eB[e] = fmaf(eA[e], sb, eB[e]);
        eA[e] *= sa;
      }
      fb[e] = none ? wb[e] : fmaf(wa[e], fb[e], wb[e]);
      fa[e] = none ? wa[e] : fa[e] * wa[e];
    }
  }
  arrive<V>(p, sh, at, at.segs - 1 - at.seg, P::start(p, at.n) + at.segs - 1, -1, chan, fa,
            fb, carry);

  float before[kRun][V];
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      before[j][e] = h[e];
      const float la2 = rate[e] * sigmoid_(rr[j].get(e));
      h[e] = fmaf(a[j][e], h[e], root_(one_minus_square(la2, a[j][e])) * sigmoid_(ri[j].get(e)) * rx[j].get(e));
    }
  }
  float K[V], total[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    K[e] = fmaf(eA[e], carry[e], eB[e]);
    total[e] = 0.f;
  }
  const __amdgpu_buffer_rsrc_t bx = tile_of<E, P::kTokens>(p.dx, row, left, p.C), br = tile_of<E, P::kTokens>(p.dr, row, left, p.C),
                               bi = tile_of<E, P::kTokens>(p.di, row, left, p.C);
#pragma unroll
  for (int j = kRun - 1; j >= 0; --j) {
    rr[j].forget();
    ri[j].forget();
    rx[j].forget();
    if constexpr (Z) {
      rz[j].forget();
      rd[j].forget();
    }
    float ox[V], orr[V], oi[V], oz[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float sr = sigmoid_(rr[j].get(e)), si = sigmoid_(ri[j].get(e)), xv = rx[j].get(e);
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
        const float zz = rz[j].get(e), sz = sigmoid_(zz);
        const float hn = fmaf(decay, hp, m * six);
        oz[e] = rd[j].get(e) * hn * sz * (1.f + zz * (1.f - sz));
      }
      total[e] += j < have ? E1 : 0.f;
    }
    Row<E, V>::store(bx, first + j * step, ox);
    Row<E, V>::store(br, first + j * step, orr);
    Row<E, V>::store(bi, first + j * step, oi);
    if (Z && p.dz) Row<E, V>::store(tile_of<E, P::kTokens>(p.dz, row, left, p.C), first + j * step, oz);
  }
  if (threadIdx.x < P::kLanes && chan && at.seg == 0 && p.dh0) {
    float last[V];
#pragma unroll
    for (int e = 0; e < V; ++e) last[e] = fmaf(fa[e], carry[e], fb[e]);
    Row<float, V>::store(p.dh0 + static_cast<int64_t>(at.n) * p.C + d, last);
  }
  // the segment's sum of E, over the runs of a wave and then over the waves
#pragma unroll
  for (int e = 0; e < V; ++e)
#pragma unroll
    for (int off = P::kLanes; off < 64; off <<= 1) total[e] += __shfl_xor(total[e], off, 64);
  __syncthreads();  // the waves' (A, B) are read
  if (at.run == 0) Row<float, V>::store(&sh.wave[at.wave][0][at.ch], total);
  __syncthreads();
  if (threadIdx.x < P::kLanes && chan) {
    float sum[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = 0.f;
#pragma unroll
    for (int w = 0; w < kGlrWaves; ++w)
#pragma unroll
      for (int e = 0; e < V; ++e) sum[e] += sh.wave[w][0][at.ch + e];
    Row<float, V>::store(p.part_lam + at.slot * p.C + d, sum);
  }
}

// dlam from the segments' sums, 64 channels a workgroup: each of 16 waves adds every
// sixteenth slot's in order, then the sixteen are added.
__global__ __launch_bounds__(1024) void glr_lam_kernel(GlrParams p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, d = blockIdx.x * 64 + lane;
  __shared__ float part[16][64];
  float sum = 0.f;
  if (d < p.C) {
#pragma unroll 8
    for (int64_t slot = wave; slot < p.slots; slot += 16) sum += p.part_lam[slot * p.C + d];
  }
  part[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && d < p.C) {
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) sum += part[w][lane];
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

// The counter and the words' marks cleared, in 16 bytes a thread.
__global__ __launch_bounds__(256) void glr_clear_kernel(uint64_t* chain, int64_t pairs) {
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at < pairs) reinterpret_cast<u32x4_t*>(chain)[at] = u32x4_t(0u);
}

template <typename E, bool BWD>
hipError_t launch(const GlrParams& p, hipStream_t s) {
  constexpr int V = glr_vec(BWD);
  static_assert(Place<V>::kTokens == glr_seg(BWD), "segments as the workspace counts them");
  const int tiles = glr_tiles(p.C);
  if (p.chained) {
    const int64_t groups = glr_slots(p.rows, p.N, glr_seg(BWD) * kGlrGroup);
    const int64_t pairs = 16 + (p.slots + groups) * p.words / 2;
    hipLaunchKernelGGL(glr_clear_kernel, dim3(static_cast<unsigned>((pairs + 255) / 256)), dim3(256), 0, s, p.chain, pairs);
  }
  const dim3 grid(static_cast<unsigned>(p.slots * tiles)), block(64 * kGlrWaves);
  if constexpr (BWD) {
    if (p.N > 0) {
      if (p.z)
        hipLaunchKernelGGL((glr_bwd_kernel<E, V, true>), grid, block, 0, s, p, tiles);
      else
        hipLaunchKernelGGL((glr_bwd_kernel<E, V, false>), grid, block, 0, s, p, tiles);
    }
    hipLaunchKernelGGL(glr_lam_kernel, dim3(static_cast<unsigned>((p.C + 63) / 64)), dim3(1024), 0, s, p);
  } else {
    if (p.z)
      hipLaunchKernelGGL((glr_fwd_kernel<E, V, true>), grid, block, 0, s, p, tiles);
    else
      hipLaunchKernelGGL((glr_fwd_kernel<E, V, false>), grid, block, 0, s, p, tiles);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_glr_fwd(const GlrParams& p, bool bf16, hipStream_t s) {
  return bf16 ? launch<uint16_t, false>(p, s) : launch<float, false>(p, s);
}

hipError_t launch_glr_bwd(const GlrParams& p, bool bf16, hipStream_t s) {
  return bf16 ? launch<uint16_t, true>(p, s) : launch<float, true>(p, s);
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
