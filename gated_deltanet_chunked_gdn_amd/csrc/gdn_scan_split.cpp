// How the selective scan is split over the time axis (host only).
#include <algorithm>

#include "gdn_layer.h"

namespace gdn {

// Packed sequences of other lengths count as so many of the longest.
static int64_t sequences(int64_t max_len, int64_t rows) {
  return max_len > 0 ? (rows + max_len - 1) / max_len : 1;
}

// Serial needs the fewest instructions; the split runs the state's part of the work
// twice, and every segment composes the ones before it.  It is taken where the channels
// alone leave SIMDs idle: segments of at least 64 tokens, as many as give every SIMD four
// waves (1024 workgroups of four; two waves, 512, for 64 states, whose registers allow no
// more).  Where that leaves fewer than half as many workgroups, the chain of tokens is
// what takes the time, and segments are shortened, to 16 tokens at least and 32 of them at
// most, for up to half as many.  Measured, bf16 (us), at least 64 / 16:
//   16 states, backward, 1 x 64 x 256    22 / 15     1 x 128 x 2048   36 / 20
//   64 states, forward,  1 x 128 x 256   39 / 18     backward 88 / 35
// but 64 states, forward, 1 x 512 x 2048 44 / 69 with 1024 workgroups of 16 tokens.
// A length between two multiples of 16 goes to the nearer one in the backward, where 16
// tokens of 32 states take 8 us alone on a CU, and up in the forward, where they take less
// than the composing of more segments (sequences of up to 374 tokens, 2 x 160 channels, 32
// states, fp32, segments of 16 / 32 tokens: backward 25 / 32 us, forward 15 / 13).
static ScanSplit split(int64_t max_len, int64_t rows, int D, int G, int N, bool nearest) {
  const int64_t want = N == 64 ? 512 : 1024;
  const int64_t groups = sequences(max_len, rows) * scan_tiles(D, G);
  int64_t segs = std::min<int64_t>((want + groups - 1) / groups, max_len / 64);
  if (segs * groups < want / 2) {
    const int64_t least = std::min<int64_t>(64, ((max_len + 31) / 32 + 15) / 16 * 16);
    segs = std::min<int64_t>((want / 2 + groups - 1) / groups, max_len / std::max<int64_t>(least, 16));
  }
  if (segs < 2) return ScanSplit{1, std::max<int64_t>(max_len, 64), 0};
  const int64_t len = nearest ? std::max<int64_t>((max_len / segs + 8) / 16 * 16, 16)
                              : ((max_len + segs - 1) / segs + 15) / 16 * 16;
  return ScanSplit{static_cast<int32_t>((max_len + len - 1) / len), len, 0};
}

ScanSplit scan_split_bwd(int64_t max_len, int64_t rows, int D, int G, int N) {
  return split(max_len, rows, D, G, N, true);
}

// The forward has a kernel with the time axis inside the workgroup, for 8 and 16 states.
// It has no second pass over the exponentials, but takes 64 tokens in 2.3 us however few
// the channels.  Measured against the split, bf16, 16 states, one sequence (us, time axis
// inside / split), for 256, 8192 and 32768 channels:
//     16 tokens  4.7 / 4.8   5.7 / 4.9    16 / 5.8   (serial then, and no wave without tokens)
//     64 tokens  4.7 / 9.5   6.3 / 11     17 / 14
//     256 tokens  11 / 13     15 / 23     55 / 59
//     512 tokens  20 / 17     28 / 40    101 / 109
//     2048 tokens 73 / 28    100 / 127   383 / 392
// and 754 / 584 for 8 x 8192 channels, where the serial kernel fills the chip.
ScanSplit scan_split_fwd(int64_t max_len, int64_t rows, int D, int G, int N) {
  const int64_t groups = sequences(max_len, rows) * scan_tiles(D, G);
  const int64_t narrow = sequences(max_len, rows) * scan_time_tiles(D, G);
  if (N <= 16 && max_len > (groups < 512 ? 16 : 64) && groups < 1024 && (max_len <= 320 || narrow >= 384))
    return ScanSplit{1, std::max<int64_t>(max_len, 64), 1};
  return split(max_len, rows, D, G, N, false);
}

}  // namespace gdn
