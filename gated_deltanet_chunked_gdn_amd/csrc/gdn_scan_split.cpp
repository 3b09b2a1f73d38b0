// How the selective scan is split over the time axis (host only).
#include <algorithm>
#include <cmath>

#include "gdn_layer.h"

namespace gdn {

// Packed sequences of other lengths count as so many of the longest.
static int64_t sequences(int64_t max_len, int64_t rows) {
  return max_len > 0 ? (rows + max_len - 1) / max_len : 1;
}

// Serial needs the fewest instructions; the split runs the state's part of the work
// twice, and every segment composes the ones before it.  It is taken where the channels
// alone leave SIMDs idle: segments of at least 64 tokens, as many as make 1024 workgroups of
// four waves (512 for 64 states, whose registers allow two waves a SIMD).  That is one round
// of workgroups in the forward with 8 and 16 states (four waves a SIMD and more), one and a
// third with 32, where the kernel of the outputs has three waves, and two in the backward,
// which has two with every number of states.  32 states with 768 instead, forward / backward,
// us: 1 x 2048 x 16384 347 -> 312 / 978 -> 1220, 1 x 16384 x 2048 389 -> 356 / 982 -> 1240,
// 1 x 2048 x 32768 629 -> 630 / 1879 -> 1883; with 512 347 -> 364, 389 -> 403, 629 -> 455 and
// 978 -> 1007, 982 -> 999, 1879 -> 1677.  Where that leaves fewer than half as many workgroups, the chain of tokens is
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
  // A segment's start is composed of the others of its sequence one after another, 0.35 us
  // (forward) or 0.4 us (backward) each; a token takes 0.2 us (forward, both kernels) or 0.35
  // us for every 16 states that the backward takes at a time.  The sum of both is least near
  // segs^2 = tokens (times those passes).  Without this bound / with it, bf16, us:
  //   64 channels, 16 states: 8192 tokens, forward 60 / 51, backward 74 / 72 (128 / 85 segments);
  //   65536 tokens, 370 / 144 and 444 / 193 (1024 / 256).  Up to 64 segments it changes nothing.
  const int64_t passes = nearest ? std::max(1, N / 16) : 1;
  segs = std::min(segs, std::max<int64_t>(64, static_cast<int64_t>(std::sqrt(static_cast<double>(max_len * passes)))));
  if (segs < 2) return ScanSplit{1, std::max<int64_t>(max_len, 64), 0};
  const int64_t len = nearest ? std::max<int64_t>((max_len / segs + 8) / 16 * 16, 16)
                              : ((max_len + segs - 1) / segs + 15) / 16 * 16;
  return ScanSplit{static_cast<int32_t>((max_len + len - 1) / len), len, 0};
}

ScanSplit scan_split_bwd(int64_t max_len, int64_t rows, int D, int G, int N) {
  return split(max_len, rows, D, G, N, true);
}

// The forward has a kernel with the time axis inside the workgroup.  It has no second pass
// over the exponentials, but takes 64 tokens in 2.3 us however few its workgroups, 512 of
// which the chip holds (a workgroup: 256 pairs of channel and state).  Measured against the
// split, bf16, one sequence (us, time axis inside / split), for W workgroups:
//          tokens    W = 64      128        256        512        1024       2048       4096
//   16 states  16   4.4 / 4.4  4.4 / 4.5  4.5 / 4.5  5.1 / 4.7  8.7 / 4.7   15 / 5.3   28 / 7.2
//              64   4.4 / 8.7  4.4 / 9.0  4.6 / 9.0  5.3 / 10   9.0 / 13    18 / 14    32 / 19
//             256    11 / 11    11 / 12    12 / 15    15 / 24    26 / 32    47 / 49    91 / 61
//             512    20 / 15    20 / 16    21 / 24    26 / 35    46 / 53    87 / 88   177 / 122
//            2048    72 / 28    73 / 40    74 / 60    87 / 104  167 / 182  329 / 324  652 / 435
//   32 states  16   4.4 / 5.4  4.4 / 5.4  4.5 / 5.4  5.2 / 5.4  8.9 / 5.5   16 / 5.7   29 / 6.9
//              64   4.5 / 11   4.5 / 11   4.7 / 11   5.5 / 11   9.3 / 14    17 / 18    34 / 19
//             512    20 / 18    21 / 24    22 / 24    26 / 35    48 / 57    92 / 93   181 / 171
//            2048    74 / 33    80 / 44    81 / 68    89 / 105  174 / 190  382 / 338  766 / 619
//   64 states  16   4.4 / 7.1  4.5 / 7.2  4.6 / 7.2  5.2 / 7.2  8.8 / 7.3   16 / 7.6   29 / 7.8
//              64   4.5 / 15   4.5 / 15   4.7 / 15   5.5 / 16   9.2 / 16    17 / 23    30 / 22
//             512    20 / 30    21 / 29    22 / 29    26 / 41    48 / 55    91 / 92   179 / 154
//            1024    38 / 37    39 / 37    40 / 45    47 / 60    90 / 95   176 / 172  347 / 297
//            2048    74 / 53    76 / 53    77 / 71    89 / 101  174 / 175  345 / 331  690 / 586
ScanSplit scan_split_fwd(int64_t max_len, int64_t rows, int D, int G, int N) {
  const int64_t wgs = sequences(max_len, rows) * scan_time_tiles(D, G, N);
  const bool fills = wgs >= 384, over = wgs >= (max_len > 256 ? 2048 : 4096);
  const bool long_enough = max_len > std::max<int64_t>(16, wgs / 32) || (N > 16 && wgs <= 512);
  if (long_enough && !over && (fills || max_len <= std::max(320, 15 * N)))
    return ScanSplit{1, std::max<int64_t>(max_len, 64), 1};
  return split(max_len, rows, D, G, N, false);
}

}  // namespace gdn
