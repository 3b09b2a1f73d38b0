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
  const void* dy;
  const float* dh_final;  // or nullptr
  void* dx;
  void* dr;
  void* di;
  void* dz;            // or nullptr
  float* part_lam;     // [segment slot][C] sums of a segment
  float* dlam;
  float* dh0;          // or nullptr
  // What the segments of a sequence tell each other (chained): a counter, then words of a
  // value and a mark that it is there.
  uint64_t* chain;     // cleared before the launch: [32] whose first counts workgroups, then
  uint64_t* whole;     // [segment slot][words] decay product and end from zero of a segment
  uint64_t* end;       // [group slot][words] state behind (backward: gradient in front of) a group
  SeqInfo seq;
  int64_t rows;        // B * T
  int64_t slots;       // segment slots
  int32_t N, C;
  int32_t words;       // C up to whole tiles
  int32_t chained;     // some sequence has several segments
  float c;
};

constexpr int kGlrRun = 8;     // tokens that a thread takes one after another
constexpr int kGlrTile = 64;   // channels of a workgroup: rows of 128 bytes (bf16)
constexpr int kGlrWaves = 4;
constexpr int kGlrGroup = 8;   // segments of a group
// Channels of a lane.
constexpr int glr_vec(bool bwd) { return bwd ? 2 : 4; }
// Tokens of a segment: the runs of a workgroup's lanes.
constexpr int glr_seg(bool bwd) { return kGlrWaves * 64 / (kGlrTile / glr_vec(bwd)) * kGlrRun; }
inline int glr_tiles(int C) { return (C + kGlrTile - 1) / kGlrTile; }
// Part c (of `len` tokens) of a sequence that starts at row bos uses slot bos / len + n + c (distinct).
inline int64_t glr_slots(int64_t rows, int64_t n, int64_t len) { return rows / len + n; }
// The segment slot of workgroup `index` of a launch over `slots` slots of `tiles` channel tiles
// (`back`: the last slot first), or -1 behind the last one: workgroups are numbered by a counter
// in the workspace, and calls that overlap and share one, against the rules, count on past their end.
__host__ __device__ inline int64_t glr_slot(int64_t index, int tiles, int64_t slots, bool back) {
  const int64_t slot = index / tiles;
  if (slot >= slots) return -1;
  return back ? slots - 1 - slot : slot;
}
hipError_t launch_glr_fwd(const GlrParams& p, bool bf16, hipStream_t s);
hipError_t launch_glr_bwd(const GlrParams& p, bool bf16, hipStream_t s);
hipError_t launch_glr_step(const GlrParams& p, bool bf16, hipStream_t s);

// ---------------------------------------------------------------------------- norm and rotation

struct RopeParams {
  const void* q;         // [tokens] rows of Hq D values, q_stride apart
  const void* k;
  const float* inv_freq; // [R / 2]
  const int32_t* pos;    // [tokens] or nullptr: the place in the row of T
  const float* wq;       // [D] or nullptr
  const float* wk;
  void* q_out;           // contiguous; backward: dq, dk
  void* k_out;
  const void* dq_out;    // backward, contiguous
  const void* dk_out;
  float* dwq;            // or nullptr
  float* dwk;
  float* part;           // backward: [workgroup][2][D] partial sums
  int64_t q_stride, k_stride;
  int64_t tokens;
  int32_t T, Hq, Hk, R;
  int32_t norm;          // gdn_rope_norm
  float eps;
  int32_t per_group;     // tokens that a workgroup takes at a time
  int32_t groups;        // workgroups
};

// Tokens of a workgroup at a time: four where that leaves every CU several workgroups.
constexpr int kRopeMost = 4;
inline int rope_tokens(int64_t tokens) { return tokens >= 1024 * kRopeMost ? kRopeMost : 1; }
// Workgroups go on to further tokens, so that the weights are loaded once and, in the
// backward, few partial sums are left.
constexpr int kRopeGroups = 1024;
inline int64_t rope_groups(int64_t tokens) {
  const int64_t n = (tokens + rope_tokens(tokens) - 1) / rope_tokens(tokens);
  return n < kRopeGroups ? n : kRopeGroups;
}
hipError_t launch_rope_fwd(const RopeParams& p, int D, bool bf16, bool interleaved, hipStream_t s);
hipError_t launch_rope_bwd(const RopeParams& p, int D, bool bf16, bool interleaved, hipStream_t s);

// ---------------------------------------------------------------------------- window attention

struct SwaParams {
  const void* q;       // rows of Hq D values, q_stride apart
  const void* k;       // rows of Hk D values
  const void* v;
  void* o;             // contiguous
  float* lse;          // [rows][Hq], or nullptr in the forward
  const void* dout;    // backward, contiguous
  void* dq;
  void* dk;
  void* dv;
  float* delta;        // backward: [rows][Hq] sums of dout o
  float* first_win;    // backward: [N][Hk][S][2][D] the first tokens' dk, dv from inside the window
  float* first_far;    // backward: [slot][Hk][S][2][D] those from queries further on, by runs of them
  int64_t q_stride, k_stride, v_stride;
  SeqInfo seq;
  int64_t rows;        // B * T
  int32_t N, Hq, Hk;
  int32_t W, S;        // W at most the longest sequence; S 0 where no window leaves a token behind
  int32_t few;         // blocks of 128 queries are too few workgroups
  int32_t few_keys;    // blocks of 128 keys are
  int32_t far;         // queries of a run for the first tokens' gradients
  float scale;
  // cache
  void* kc;            // [N][slots][Hk][D]
  void* vc;
  const int32_t* lens; // step: tokens before this one, negative: an idle place
  int32_t slots;       // S + W
  int32_t splits;      // step: runs of slots, a workgroup each
  int32_t run;         // step: slots of a run
  float* part;         // step: [split][N][Hq] (maximum, sum), then [split][N][Hq][D] values
};
constexpr int kSwaQueries = 128;  // queries of a workgroup
constexpr int kSwaKeys = 128;     // keys of a workgroup of the backward
// Run c (of `far` queries) of a sequence that starts at row bos uses slot bos / far + n + c (distinct).
inline int64_t swa_far_slots(int64_t rows, int64_t n, int64_t far) { return rows / far + n; }
// Blocks of `each` rows that a launch counts: a dense sequence's as many as it needs, those of
// packed sequence n from cu[n] / each + n on (distinct; some are no sequence's).
inline int64_t swa_slots(const SwaParams& p, int64_t rows, int64_t each) {
  return p.seq.cu ? rows / each + p.N : p.N * ((p.seq.T + each - 1) / each);
}
// The workgroups of a launch: chunks of slots after each other, each chunk's key heads, slots and
// (of queries) a key head's query heads, the last the fastest, an eighth on each XCD.  Dense
// sequences are one chunk.  Packed ones, whose blocks of unlike work lie in rows, come in chunks of
// 16 slots or fewer, so that every XCD has some of each.  Forward, 16 / 4 heads of 128, window 1024, bf16, us, by
// chunks of 4, 8, 16, 32 and 64: 2048 tokens in two sequences 34, 34, 34, 40, 37; 10240 in six 101, 102,
// 105, 106, 100; 4096 in nine 48, 45, 44, 46, 50; training, 8 / 1 heads of 64, fp32, 8192 tokens in
// six 454, 477, 458, 521, 524.
struct SwaWork {
  int32_t slots, chunk;  // slots of a chunk
  int32_t heads;         // query heads of a key head, or 1
  int32_t share;         // workgroups of an XCD in a chunk
};
struct SwaGrid {
  dim3 grid;
  SwaWork work;
};
inline SwaGrid swa_grid(const SwaParams& p, int64_t each, int heads, int z = 1) {
  const int64_t slots = swa_slots(p, p.rows, each);
  const int64_t chunks = p.seq.cu ? (slots + 15) / 16 : 1, chunk = (slots + chunks - 1) / chunks;
  const int64_t share = (chunk * p.Hk * heads + 7) / 8, total = 8 * chunks * share;
  // a grid's axis has up to 2^32 threads
  const int64_t y = (total + (1 << 22) - 1) >> 22, x = ((total + y - 1) / y + 7) / 8 * 8;
  return SwaGrid{dim3(static_cast<unsigned>(x), static_cast<unsigned>(y), static_cast<unsigned>(z)),
                 SwaWork{static_cast<int32_t>(slots), static_cast<int32_t>(chunk), heads, static_cast<int32_t>(share)}};
}
hipError_t launch_swa_fwd(const SwaParams& p, int D, bool bf16, hipStream_t s);
hipError_t launch_swa_bwd(const SwaParams& p, int D, bool bf16, hipStream_t s);
hipError_t launch_swa_fill(const SwaParams& p, int D, bool bf16, hipStream_t s);
hipError_t launch_swa_step(const SwaParams& p, int D, bool bf16, hipStream_t s);

}  // namespace gdn
