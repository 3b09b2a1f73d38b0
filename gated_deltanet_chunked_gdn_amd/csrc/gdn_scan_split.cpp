// How the selective scan is split over the time axis (host only).
#include <algorithm>

#include "gdn_layer.h"

namespace gdn {

// Serial needs the fewest instructions; the split runs the state's part of the work
// twice.  It is taken where the channels alone leave SIMDs idle: segments of at least
// 64 tokens, as many as give every SIMD four waves (1024 workgroups of four).
// Measured, forward, bf16, 16 states: 2 x 2048 x 4096 137 us, 160 us with two waves;
// 1 x 1024 x 1024 23 us, 36 us with segments of 128 tokens at least.
ScanSplit scan_split(int64_t max_len, int64_t nseq, int D, int G) {
  const int64_t groups = nseq * scan_tiles(D, G);
  const int64_t segs = std::min<int64_t>((1024 + groups - 1) / groups, max_len / 64);
  if (segs < 2) return ScanSplit{1, std::max<int64_t>(max_len, 64)};
  const int64_t len = ((max_len + segs - 1) / segs + 63) / 64 * 64;
  return ScanSplit{static_cast<int32_t>((max_len + len - 1) / len), len};
}

}  // namespace gdn
