// How the selective scan is split over the time axis (host only).
#include <algorithm>

#include "gdn_layer.h"

namespace gdn {

static int64_t sequences(int64_t max_len, int64_t rows) {
  return max_len > 0 ? (rows + max_len - 1) / max_len : 1;
}

// Serial needs the fewest instructions; the split runs the state's part of the work
// twice.  It is taken where the channels alone leave SIMDs idle: segments of at least
// 64 tokens, as many as give every SIMD four waves (1024 workgroups of four).
// Measured, forward, bf16, 16 states: 2 x 2048 x 4096 137 us, 160 us with two waves;
// 1 x 1024 x 1024 23 us, 36 us with segments of 128 tokens at least.
ScanSplit scan_split_bwd(int64_t max_len, int64_t rows, int D, int G) {
  // packed sequences of other lengths count as so many of the longest
  const int64_t groups = sequences(max_len, rows) * scan_tiles(D, G);
  const int64_t segs = std::min<int64_t>((1024 + groups - 1) / groups, max_len / 64);
  if (segs < 2) return ScanSplit{1, std::max<int64_t>(max_len, 64), 0};
  const int64_t len = ((max_len + segs - 1) / segs + 63) / 64 * 64;
  return ScanSplit{static_cast<int32_t>((max_len + len - 1) / len), len, 0};
}

// The forward has a kernel with the time axis inside the workgroup, for 8 and 16 states.
// It has no second pass over the exponentials, but takes 64 tokens in 2.3 us however few
// the channels.  Measured against the split, bf16, 16 states, one sequence (us, time axis
// inside / split), for 1024, 8192 and 32768 channels:
//     32 tokens and less: the split's kernel, which is serial then, wastes no waves
//     128 tokens   7 / 19      9 / 20      30 / 34
//     512 tokens  20 / 21     29 / 40     101 / 109
//     2048 tokens 74 / 30    102 / 129    383 / 392
// and 754 / 584 for 8 x 8192 channels, where the serial kernel fills the chip.
ScanSplit scan_split_fwd(int64_t max_len, int64_t rows, int D, int G, int N) {
  const int64_t groups = sequences(max_len, rows) * scan_tiles(D, G);
  const int64_t narrow = sequences(max_len, rows) * scan_time_tiles(D, G);
  if (N <= 16 && max_len > 32 && groups < 1024 && (max_len <= 384 || narrow >= 384))
    return ScanSplit{1, std::max<int64_t>(max_len, 64), 1};
  return scan_split_bwd(max_len, rows, D, G);
}

}  // namespace gdn
