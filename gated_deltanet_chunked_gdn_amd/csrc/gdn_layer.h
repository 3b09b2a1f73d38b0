// Host-visible kernel parameter blocks and launchers of the layer operators: the
// single-token step of the delta rule, the short causal convolution, the selective
// scan (internal).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_internal.h"

namespace gdn {

struct StepParams {
  const void* q;      // [B][H][Dk]
  const void* k;
  const void* v;      // [B][H][Dv]
  const float* g;     // [B][H], or [B][H][Dk] (channel)
  const float* beta;  // [B][H]
  float* S;           // [B][H][Dk][Dv], updated in place
  void* o;            // [B][H][Dv]
  int64_t heads;      // B * H
  int32_t Dv;
  float scale;
};
hipError_t launch_step(const StepParams& p, int Dk, bool bf16, bool channel, hipStream_t s);

struct ConvParams {
  const void* x;
  const float* weight;  // [C][W]
  const float* bias;    // [C] or nullptr
  const void* state0;   // [N][W-1][C] or nullptr
  void* y;
  void* state_final;    // [N][W-1][C] or nullptr
  const void* dy;
  const void* dstate_final;  // or nullptr
  void* dx;
  float* dweight;
  float* dbias;         // or nullptr
  void* dstate0;        // or nullptr
  float* ws;            // backward: [token block][W + 1][C] partial sums
  SeqInfo seq;
  int64_t rows;         // B * T
  int32_t N, C;
  int32_t silu;
};
// Token blocks of the backward's partial sums.
constexpr int kConvBwdRows = 512;
inline int64_t conv_bwd_blocks(int64_t rows) { return (rows + kConvBwdRows - 1) / kConvBwdRows; }
hipError_t launch_conv_fwd(const ConvParams& p, int W, bool bf16, hipStream_t s);
hipError_t launch_conv_bwd(const ConvParams& p, int W, bool bf16, hipStream_t s);
// state in p.state_final, updated in place
hipError_t launch_conv_step(const ConvParams& p, int W, bool bf16, hipStream_t s);

struct ScanParams {
  const void* u;
  const void* dt;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* Dskip;
  const void* z;
  const float* dt_bias;
  const float* h0;
  void* y;
  float* h_final;
  float* saved;         // [block slot][D][N] states before every block, or nullptr
  // segments over the time axis: `segs` runs of `seg_len` tokens (a multiple of
  // kScanBlock) of every sequence
  float* seg_end;       // [slot][D][N], slot bos / seg_len + n + segment (as the kept states)
  float* seg_sum;       // [slot][D]: sums of delta
  SeqInfo seq;
  int32_t nseq, D, G;
  int32_t softplus;
  int32_t segs;
  int64_t seg_len;
  int32_t in_time;      // forward: the time axis inside the workgroup (segs == 1)
  // backward
  const void* dy;
  const float* dh_final;
  void* du;
  void* ddt;
  float* dA;
  void* dBm;
  void* dCm;
  float* dDskip;
  void* dz;
  float* ddt_bias;
  float* dh0;
  float* part_bc;       // [channel tile][row][2][N] partial dB, dC
  float* part_a;        // [slot][D][N + 2] partial dA, dDskip, ddt_bias
  int64_t parts;        // slots of segments: rows / seg_len + sequences
  int64_t rows;         // B * T
};

constexpr int kScanTile = 64;     // channels per workgroup
constexpr int kScanBlock = 16;    // tokens between two kept states
// Kept-state slots: block c of a sequence that starts at row bos uses slot
// bos / block + n + c (distinct, as chunk_slots).
inline int64_t scan_slots(int64_t rows, int64_t nseq) { return rows / kScanBlock + nseq + 1; }
inline int scan_tiles(int D, int G) { return G * ((D / G + kScanTile - 1) / kScanTile); }
// Segments of the longest sequence, of max_len of all the rows, and their length; `in_time`: the
// forward's kernel with the time axis inside the workgroup instead.
struct ScanSplit {
  int32_t segs;
  int64_t len;
  int32_t in_time;
};
ScanSplit scan_split_fwd(int64_t max_len, int64_t rows, int D, int G, int N);
ScanSplit scan_split_bwd(int64_t max_len, int64_t rows, int D, int G, int N);
hipError_t launch_scan_fwd(const ScanParams& p, int N, bool bf16, hipStream_t s);
// Channels of a workgroup of that kernel, and workgroups of a sequence.
constexpr int scan_time_channels(int N) { return N <= 16 ? 16 : 256 / N; }
inline int scan_time_tiles(int D, int G, int N) {
  return G * ((D / G + scan_time_channels(N) - 1) / scan_time_channels(N));
}
hipError_t launch_scan_time(const ScanParams& p, int N, bool bf16, hipStream_t s);
hipError_t launch_scan_bwd(const ScanParams& p, int N, bool bf16, hipStream_t s);
// state in p.h_final, updated in place
hipError_t launch_scan_step(const ScanParams& p, int N, bool bf16, hipStream_t s);

}  // namespace gdn
