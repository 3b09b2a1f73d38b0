// Host-visible kernel parameter blocks and launchers of the operators that hybrid
// models put next to the delta rule: the gated linear recurrence, the norm and rotation
// of queries and keys, and attention over a sliding window (internal).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_internal.h"

namespace gdn {

// ---------------------------------------------------------------------------- recurrence

struct GlrParams {
  const void* x;       // [rows][C]
  const void* r;
  const void* i;
  const float* lam;    // [C]
  const void* z;       // or nullptr
  const float* h0;     // [N][C] or nullptr
  void* y;
  float* h_final;      // [N][C] or nullptr; the step's state, updated in place
  float* saved;        // [run slot][C] states before every run of kGlrRun tokens, or nullptr
  float* seg;          // [part][2][C] decay product and end state of every segment
  const void* dy;
  const float* dh_final;  // or nullptr
  void* dx;
  void* dr;
  void* di;
  void* dz;            // or nullptr
  float* part_lam;     // [part][C] sums of a segment
  float* dlam;
  float* dh0;          // or nullptr
  SeqInfo seq;
  int64_t rows;        // B * T
  int32_t N, C;
  int32_t segs;        // segments of the longest sequence, of seg_len tokens
  int32_t waves;       // waves of a workgroup (1, 2, 4 or 8)
  int64_t seg_len;
  float c;
};

constexpr int kGlrRun = 8;    // tokens that a thread takes one after another
constexpr int kGlrTile = 32;  // channels of a workgroup
inline int glr_tiles(int C) { return (C + kGlrTile - 1) / kGlrTile; }
// Run c of a sequence that starts at row bos uses slot bos / run + n + c (distinct).
inline int64_t glr_slots(int64_t rows, int64_t n) { return rows / kGlrRun + n + 1; }
inline int64_t glr_parts(int64_t rows, int64_t n, int64_t seg_len) { return rows / seg_len + n; }
hipError_t launch_glr_fwd(const GlrParams& p, bool bf16, hipStream_t s);
hipError_t launch_glr_bwd(const GlrParams& p, bool bf16, hipStream_t s);
hipError_t launch_glr_step(const GlrParams& p, bool bf16, hipStream_t s);

}  // namespace gdn
