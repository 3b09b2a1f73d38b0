// Device helpers of the window attention's kernels: tiles of rows in LDS, operands of the
// matrix instructions, the window's mask.
//
// Products are formed on 16x16 tiles.  What a lane (c = lane % 16, g = lane / 16) gives to
// one "step" of a product is 16 bytes: bf16 8 values of the reduction (one instruction over
// 32), fp32 4 values (four instructions over 16).  The order of the reduction is free as long as both
// operands share it, and two orders are used:
//   * along a row of values (d): column COLS step + EPP g + e; both operands are pieces of
//     16 bytes of rows, from memory or from LDS;
//   * along rows (keys or queries): row 16 b + 4 g + r of the step's blocks b, the rows that
//     an accumulator holds in lane (c, g), so scores go from the accumulators of one product
//     into the operand of the next without leaving their registers.  The other operand
//     comes from LDS by transposing reads (bf16) or down a column (fp32).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_chunk_common.h"
#include "gdn_device.h"
#include "gdn_hybrid.h"

namespace gdn {
namespace swa {

using chunk::u32x4_t;
constexpr float kLog2e = chunk::kLog2e;
constexpr float kLn2 = 0.6931471805599453f;

// A tile of rows of D values in LDS.  The piece of 16 bytes u of row t stands at u ^ swizzle(t).
// LDS serves 256 bytes at a time.  Along rows those are 16 lanes' pieces, of rows 0-3 and
// 12-15 from one lane group and 4-11 from the next; down the rows (bf16) two lane groups', of
// rows 0-7 or 8-15 and two neighbouring pieces.  So the eight pairs of pieces go to rows 0-7
// in order and again to rows 12-15 and 8-11 with the two swapped, which keeps both ways apart
// (half as many pieces: rows two by two).  In fp32 four lane groups read one row each of
// four, 16 bytes a lane's four: rows one piece apart.
template <typename E, int D>
struct Tile {
  static constexpr int kEpp = 16 / static_cast<int>(sizeof(E));  // values of a piece
  static constexpr int kPieces = D / kEpp;                       // pieces of a row: 8, 16 or 32
  static __device__ __forceinline__ int swizzle(int row) {
    if (sizeof(E) == 4) return row & 15;
    constexpr int half = kPieces / 2;
    const int e = kPieces == 8 ? row >> 1 : row;
    return (((e & (half - 1)) << 1) | ((e / half) & 1)) ^ (e & half);
  }
  static __device__ __forceinline__ int at(int row, int piece) { return row * D + ((piece ^ swizzle(row)) * kEpp); }
};

struct MmaBf16 {
  using elem = uint16_t;
  static constexpr int kCols = 32;  // columns of a step along a row
  static constexpr int kBlocks = 2; // 16-row blocks of a step along rows
  static __device__ __forceinline__ f32x4_t mma(u32x4_t a, u32x4_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  }
  // Rounding to bf16: the operands of the second products are probabilities and the scores'
  // gradients, off by at most 2^-8 of each, as the inputs they are multiplied with are.  With `rest`
  // as a second product the error of a prompt's o against 64 bits is 1.6e-3 for 2.1e-3, and the
  // forward of 2 x 4096 tokens, 16 heads of 128, window 1024, takes 131 us for 98: the prompt and
  // the backward do without it, the step, which waits for memory, does not.
  static __device__ __forceinline__ u32x4_t operand(const f32x4_t* acc) {
    return u32x4_t{pack_bf16x2(acc[0][0], acc[0][1]), pack_bf16x2(acc[0][2], acc[0][3]), pack_bf16x2(acc[1][0], acc[1][1]),
                   pack_bf16x2(acc[1][2], acc[1][3])};
  }
  // What that rounding leaves (exact in fp32), rounded in turn: as the operand of a second product
  // it leaves 2^-16 of each value.
  static __device__ __forceinline__ u32x4_t rest(const f32x4_t* acc, u32x4_t op) {
    f32x4_t left[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      left[i >> 1][2 * (i & 1)] = acc[i >> 1][2 * (i & 1)] - __uint_as_float(op[i] << 16);
      left[i >> 1][2 * (i & 1) + 1] = acc[i >> 1][2 * (i & 1) + 1] - __uint_as_float(op[i] & 0xffff0000u);
    }
    return operand(left);
  }
  // Columns d0 .. d0 + 15 of the 32 rows from row0 on, as the operand whose lane (c, g) holds
  // column d0 + c of rows 4 g + 0..3 of both blocks.  ds_read_b64_tr_b16: within 16 lanes, lane s names
  // row s / 4, columns 4 (s % 4) .. + 3, and lane i receives column i of the four rows.
  template <int D>
  static __device__ __forceinline__ u32x4_t read_tr(const elem* tile, int row0, int d0, int lane) {
    const int s = lane & 15, row = row0 + 4 * (lane >> 4) + (s >> 2);
    const elem* const p = tile + Tile<elem, D>::at(row, (d0 >> 3) + ((s & 3) >> 1)) + 4 * (s & 1);
    const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(p));
    const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(p + 16 * D));
    typedef short i16x8_t __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(u32x4_t, static_cast<i16x8_t>(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)));
  }
};

struct MmaF32 {
  using elem = float;
  static constexpr int kCols = 16;
  static constexpr int kBlocks = 1;
  static __device__ __forceinline__ f32x4_t mma(u32x4_t a, u32x4_t b, f32x4_t c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ u32x4_t operand(const f32x4_t* acc) { return __builtin_bit_cast(u32x4_t, acc[0]); }
  template <int D>
  static __device__ __forceinline__ u32x4_t read_tr(const elem* tile, int row0, int d0, int lane) {
    const int col = d0 + (lane & 15);
    u32x4_t v;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      v[r] = __float_as_uint(tile[Tile<elem, D>::at(row0 + 4 * (lane >> 4) + r, col >> 2) + (col & 3)]);
    return v;
  }
};

// A row's operand: 16 bytes of row `row0 + lane % 16`, step `s` along it.
template <typename Op, int D>
__device__ __forceinline__ u32x4_t read_row(const typename Op::elem* tile, int row0, int s, int lane) {
  return *reinterpret_cast<const u32x4_t*>(tile + Tile<typename Op::elem, D>::at(row0 + (lane & 15), 4 * s + (lane >> 4)));
}
template <typename Op>
__device__ __forceinline__ u32x4_t load_row(const typename Op::elem* row, int s, int lane) {
  constexpr int epp = 16 / static_cast<int>(sizeof(typename Op::elem));
  return *reinterpret_cast<const u32x4_t*>(row + s * Op::kCols + epp * (lane >> 4));
}

// ROWS rows of D values from memory to a tile, by 256 threads, without a stop in registers: a
// wave's load puts its lanes' 16 bytes one behind another into LDS, so the lane takes the
// piece that belongs where it stands.  Rows are read through a resource that ends with the
// last one, so those behind it come as zeros.  Who reads the tile waits for `landed` and then
// for the workgroup.
template <typename E, int D, int ROWS>
struct Stage {
  using T = Tile<E, D>;
  static constexpr int kRows = 64 / T::kPieces;                    // rows of a wave's load
  static constexpr int kN = (ROWS + 4 * kRows - 1) / (4 * kRows);  // loads of a wave
  static constexpr int kKinds = 4 * kRows % 16 && T::kPieces > 8 ? 2 : 1;  // swizzles of a lane's rows
  uint32_t off[kKinds];  // of this lane's piece in the first loads
  uint32_t step, wave;   // bytes from row to row
  // `stride` values from row to row
  __device__ __forceinline__ explicit Stage(int64_t stride, int thread = threadIdx.x) {
    wave = __builtin_amdgcn_readfirstlane(thread >> 6);
    step = static_cast<uint32_t>(stride) * sizeof(E);
    const int lane = thread & 63;
#pragma unroll
    for (int i = 0; i < kKinds; ++i) {
      const int row = (4 * i + wave) * kRows + lane / T::kPieces;
      off[i] = row * step + ((lane % T::kPieces) ^ T::swizzle(row)) * 16;
    }
  }
  // `rows` rows (any number; those of the tile count) from `base` on
  __device__ __forceinline__ void load(E* tile, const E* base, int rows) const {
    const int n = min(rows, ROWS);
    // as chunk::buffer_rsrc
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    const u32x4_t r = {static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32) & 0xffffu,
                       n > 0 ? (n - 1) * step + D * static_cast<uint32_t>(sizeof(E)) : 0u, 0x00020000u};
    const uint32_t to = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)tile)) + wave * 1024;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if (ROWS % (4 * kRows) && (4 * i + wave) * kRows >= ROWS) break;  // fewer rows than four waves take
      const uint32_t from = off[i % kKinds] + i / kKinds * kKinds * 4 * kRows * step;
      // In assembly, since the compiler would wait for the next tile's loads before it reads this
      // one: it cannot tell the two buffers apart.  Nothing is written to a register; M0 names
      // the place in LDS (a wait state between its write and the load).  The compiler keeps
      // nothing in M0 from one instruction to another; the kernels here have no other use of it.
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to + i * 4096), "v"(from), "s"(r) : "memory");
    }
  }
};
// This wave's loads have arrived (vmcnt 0), those above among them, which the compiler does not count.
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// At the head of a branch that few tiles take: keeps the compiler from computing it always
// and selecting (it does not move what stands behind this).
__device__ __forceinline__ void seldom() { __builtin_amdgcn_wave_barrier(); }

// Query i sees key j: no later one, and of the earlier ones the last W (itself among them)
// and the first S.
__device__ __forceinline__ bool sees(int i, int j, int W, int S) { return j <= i && (j > i - W || j < S); }

// Infinities and NaN.  A row that some columns of a product do not see stands there with
// zeros, and zero times what is not finite would be NaN.  So where a tile is not seen whole,
// such values are taken out of it (clean), and whoever has seen one becomes NaN (spoil).
__device__ __forceinline__ bool odd_(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }
// The values of a register that are not finite to zero.
template <typename E>
__device__ __forceinline__ uint32_t clean_(uint32_t w) {
  if constexpr (sizeof(E) == 4) return (w & 0x7f800000u) == 0x7f800000u ? 0u : w;
  return w & (((w & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) | ((w & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u));
}
template <typename E>
__device__ __forceinline__ u32x4_t clean_(u32x4_t v) {
  return u32x4_t{clean_<E>(v[0]), clean_<E>(v[1]), clean_<E>(v[2]), clean_<E>(v[3])};
}
// By all 256 threads: whether this thread's part of a tile holds such values.
template <typename E, int SIZE>
__device__ __forceinline__ bool odd_part(const E* tile) {
  bool mine = false;
#pragma unroll
  for (int i = 0; i < SIZE * static_cast<int>(sizeof(E)) / 4096; ++i) {
    const u32x4_t v = reinterpret_cast<const u32x4_t*>(tile)[256 * i + threadIdx.x], w = clean_<E>(v);
    mine |= w[0] != v[0] || w[1] != v[1] || w[2] != v[2] || w[3] != v[3];
  }
  return mine;
}
template <typename E, int SIZE>
__device__ __forceinline__ void clean_part(E* tile) {
#pragma unroll 1
  for (int i = 0; i < SIZE * static_cast<int>(sizeof(E)) / 4096; ++i) {
    u32x4_t* const v = reinterpret_cast<u32x4_t*>(tile) + 256 * i + threadIdx.x;
    *v = clean_<E>(*v);
  }
}
// The sums of those columns that see row `row`, where its value is not finite.  `values`: the
// row, whole; column u of this lane sees it if sees[u].
template <typename E, int ND, int CT>
__device__ __forceinline__ void spoil(f32x4_t (*acc)[CT], const E* values, const bool* sees, int lane) {
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const bool bad = odd_(IoT<E>::ld(values + 16 * d + 4 * (lane >> 4) + r));
#pragma unroll
      for (int u = 0; u < CT; ++u) acc[d][u][r] = bad && sees[u] ? __uint_as_float(0x7fc00000u) : acc[d][u][r];
    }
}

// What the workgroup works on: workgroups x, x + 8, ... share an XCD and its L2.
struct Item {
  int hk, slot, head;  // head: of the key head's; slot: -1 for no work
};
__device__ __forceinline__ Item item_of(const SwaParams& p, const SwaWork& w) {
  const int x = blockIdx.y * gridDim.x + blockIdx.x, k = x >> 3, chunk = k / w.share;
  const int at = (x & 7) * w.share + k - chunk * w.share, hk = at / (w.heads * w.chunk), rest = at - hk * w.heads * w.chunk;
  const int in = rest / w.heads, slot = chunk * w.chunk + in;
  return Item{hk, hk < p.Hk && slot < w.slots ? slot : -1, rest - in * w.heads};
}

// The sequence of a slot (swa_slots) and its block there.
struct Spot {
  int n, block, len;
  int64_t bos;
};
__device__ __forceinline__ Spot spot(const SwaParams& p, int slot, int each) {
  Spot s;
  int64_t len;
  if (p.seq.cu) {
    // The last sequence whose slots begin at or before this one, by a whole wave: 64 places at a time.
    int lo = 0, hi = p.N;
    while (hi - lo > 1) {
      const int step = (hi - lo + 63) >> 6, mid = lo + (threadIdx.x & 63) * step;
      const bool in = mid < hi && p.seq.cu[mid] / each + mid <= slot;  // the first is in
      const int at = lo + (63 - __builtin_clzll(__ballot(in))) * step;
      hi = min(hi, at + step);
      lo = at;
    }
    s.n = lo;
    chunk::seq_range(p.seq, lo, s.bos, len);
    s.block = slot - static_cast<int>(s.bos / each) - lo;
  } else {
    const int blocks = (p.seq.T + each - 1) / each;
    s.n = slot / blocks;
    s.block = slot - s.n * blocks;
    chunk::seq_range(p.seq, s.n, s.bos, len);
  }
  s.len = static_cast<int>(len);
  return s;
}

}  // namespace swa
}  // namespace gdn
