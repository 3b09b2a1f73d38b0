// C ABI of the layer operators (gdn_step, gdn_conv_*, gdn_scan_*): argument
// validation, workspace sizing and dispatch.  Every check runs on the host before
// the first launch (see include/gdn.h).
#include "gdn.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gdn_abi_check.h"
#include "gdn_layer.h"

namespace {

using gdn::check::check_seqs;
using gdn::check::check_tensors;
using gdn::check::hip_status;
using gdn::check::up256;

// ---------------------------------------------------------------------------- step

gdn_status step(const gdn_problem* p, const void* q, const void* k, const void* v, const float* g,
                const float* beta, float* S, void* o, void* stream, bool channel) {
  // the problem's own checks are those of gdn_recurrent_ref
  size_t unused = 0;
  gdn_status st = gdn_workspace_size(p, GDN_PASS_RECURRENT_FWD, &unused);
  if (st != GDN_OK) return st;
  if (p->T != 1 || p->cu_seqlens_host) return GDN_ERR_SHAPE;
  // workgroups of 256 threads, up to Dv / 32 of them a head, counted in 32-bit threads
  if (static_cast<int64_t>(p->B) * p->H * ((p->Dv + 31) / 32) >= 1 << 24) return GDN_ERR_UNSUPPORTED;
  const size_t io = p->io_dtype == GDN_BF16 ? 2 : 4;
  const size_t heads = static_cast<size_t>(p->B) * p->H;
  const size_t nk = heads * p->Dk, nv = heads * p->Dv;
  st = check_tensors({{q, nk * io, 16, true}, {k, nk * io, 16, true}, {v, nv * io, 16, true},
                      {g, (channel ? nk : heads) * 4, 4, true}, {beta, heads * 4, 4, true}},
                     {{S, nk * p->Dv * 4, 16, true}, {o, nv * io, 16, true}});
  if (st != GDN_OK || heads == 0) return st;
  gdn::StepParams sp{};
  sp.q = q; sp.k = k; sp.v = v; sp.g = g; sp.beta = beta; sp.S = S; sp.o = o;
  sp.heads = static_cast<int64_t>(heads); sp.Dv = p->Dv; sp.scale = p->scale;
  return hip_status(gdn::launch_step(sp, p->Dk, io == 2, channel, static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------------------- convolution

struct ConvSize {
  size_t io = 0, values = 0, state = 0, weight = 0, bias = 0, ws = 0;
  int64_t rows = 0;
};

gdn_status check_conv(const gdn_conv_problem* p, ConvSize* c) {
  if (!p) return GDN_ERR_NULL;
  if (p->io_dtype != GDN_FP32 && p->io_dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (p->B < 0 || p->T < 0 || p->C <= 0 || p->W <= 0 || p->num_seqs < 0) return GDN_ERR_SHAPE;
  if (p->C % 8 != 0 || p->C > 1 << 20 || p->W < 2 || p->W > 4) return GDN_ERR_UNSUPPORTED;
  if (p->activation != GDN_ACT_NONE && p->activation != GDN_ACT_SILU) return GDN_ERR_UNSUPPORTED;
  int64_t max_len = 0;
  const gdn_status st = check_seqs(p, &max_len);
  if (st != GDN_OK) return st;
  c->io = p->io_dtype == GDN_BF16 ? 2 : 4;
  c->rows = static_cast<int64_t>(p->B) * p->T;
  if (c->rows > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  // A launch counts its threads in 32 bits.  Vectors of V channels: the forward takes one
  // thread for 8 rows of 4 channels (for 2 rows where those are below 2^16) and one for each
  // vector of the kept rows; the step and the backward's last kernel one for each vector of
  // the sequences, the latter (W + 1) C more.  2^23 covers what is rounded up, those (W + 1) C
  // (at most 5 2^20) and the threads of two rows (at most 2^18 + 2^17 more).
  const int64_t vec = 16 / static_cast<int64_t>(c->io);
  const int64_t threads = c->rows * p->C / 32 + static_cast<int64_t>(p->num_seqs) * (p->W - 1) * (p->C / vec);
  if (threads > (INT64_C(1) << 32) - (1 << 23)) return GDN_ERR_UNSUPPORTED;
  c->values = static_cast<size_t>(c->rows) * p->C * c->io;
  c->state = static_cast<size_t>(p->num_seqs) * (p->W - 1) * p->C * c->io;
  c->weight = static_cast<size_t>(p->C) * p->W * 4;
  c->bias = static_cast<size_t>(p->C) * 4;
  c->ws = static_cast<size_t>(gdn::conv_bwd_blocks(c->rows)) * p->C * (p->W + 1) * 4;
  return GDN_OK;
}

gdn::ConvParams conv_params(const gdn_conv_problem* p, const ConvSize& c, const void* x, const float* weight,
                            const float* bias) {
  gdn::ConvParams cp{};
  cp.x = x; cp.weight = weight; cp.bias = bias;
  cp.seq = gdn::SeqInfo{p->cu_seqlens_dev, p->T};
  cp.rows = c.rows; cp.N = p->num_seqs; cp.C = p->C;
  cp.silu = p->activation == GDN_ACT_SILU;
  return cp;
}

// ---------------------------------------------------------------------------- scan

struct ScanSize {
  size_t io = 0, values = 0, bc = 0, a = 0, chan = 0, state = 0;
  int64_t rows = 0;
  gdn::ScanSplit split{1, 0, 0};
  int64_t parts = 0;                     // slots of segments
  size_t saved = 0;                      // kept states
  size_t seg_end = 0, seg_sum = 0;       // segment states and sums of delta (segs > 1)
  size_t part_bc = 0, part_a = 0;        // backward: partial sums
};

gdn_status check_scan(const gdn_scan_problem* p, bool bwd, ScanSize* c) {
  if (!p) return GDN_ERR_NULL;
  if (p->io_dtype != GDN_FP32 && p->io_dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (p->B < 0 || p->T < 0 || p->D <= 0 || p->N <= 0 || p->G <= 0 || p->num_seqs < 0 || p->D % p->G != 0)
    return GDN_ERR_SHAPE;
  if (p->N != 8 && p->N != 16 && p->N != 32 && p->N != 64) return GDN_ERR_UNSUPPORTED;
  if (p->D / p->G % 8 != 0) return GDN_ERR_UNSUPPORTED;
  int64_t max_len = 0;
  const gdn_status st = check_seqs(p, &max_len);
  if (st != GDN_OK) return st;
  c->io = p->io_dtype == GDN_BF16 ? 2 : 4;
  c->rows = static_cast<int64_t>(p->B) * p->T;
  // threads (two values of dBm or dCm each, in the backward) are counted in 32 bits
  if (c->rows > INT32_MAX || c->rows * p->G * p->N >= INT64_C(1) << 32 || p->D > 1 << 20) return GDN_ERR_UNSUPPORTED;
  c->values = static_cast<size_t>(c->rows) * p->D * c->io;
  c->bc = static_cast<size_t>(c->rows) * p->G * p->N * c->io;
  c->a = static_cast<size_t>(p->D) * p->N * 4;
  c->chan = static_cast<size_t>(p->D) * 4;
  c->state = static_cast<size_t>(p->num_seqs) * c->a;
  if (p->num_seqs == 0) return GDN_OK;
  c->split = bwd ? gdn::scan_split_bwd(max_len, c->rows, p->D, p->G, p->N)
                 : gdn::scan_split_fwd(max_len, c->rows, p->D, p->G, p->N);
  c->parts = c->rows / c->split.len + p->num_seqs;
  const size_t parts = static_cast<size_t>(c->parts);
  c->saved = static_cast<size_t>(gdn::scan_slots(c->rows, p->num_seqs)) * c->a;
  if (c->split.segs > 1) {
    c->seg_end = up256(parts * c->a);
    c->seg_sum = up256(parts * c->chan);
  }
  c->part_bc = up256(static_cast<size_t>(gdn::scan_tiles(p->D, p->G) / p->G) * c->rows * p->G * 2 * p->N * 4);
  c->part_a = parts * p->D * (p->N + 2) * 4;
  return GDN_OK;
}

gdn::ScanParams scan_params(const gdn_scan_problem* p, const ScanSize& c, const void* u, const void* dt,
                            const float* A, const void* Bm, const void* Cm, const float* Dskip, const void* z,
                            const float* dt_bias) {
  gdn::ScanParams sp{};
  sp.u = u; sp.dt = dt; sp.A = A; sp.Bm = Bm; sp.Cm = Cm; sp.Dskip = Dskip; sp.z = z; sp.dt_bias = dt_bias;
  sp.seq = gdn::SeqInfo{p->cu_seqlens_dev, p->T};
  sp.nseq = p->num_seqs; sp.D = p->D; sp.G = p->G;
  sp.softplus = p->dt_softplus != 0;
  sp.segs = c.split.segs; sp.seg_len = c.split.len; sp.in_time = c.split.in_time;
  sp.parts = c.parts;
  sp.rows = c.rows;
  return sp;
}

void set_segments(gdn::ScanParams* sp, const ScanSize& c, void* ws) {
  if (c.split.segs <= 1) return;
  sp->seg_end = static_cast<float*>(ws);
  sp->seg_sum = reinterpret_cast<float*>(static_cast<char*>(ws) + c.seg_end);
}

gdn_status scan_fwd(const gdn_scan_problem* p, const void* u, const void* dt, const float* A, const void* Bm,
                    const void* Cm, const float* Dskip, const void* z, const float* dt_bias, const float* h0,
                    void* y, float* h_final, bool save, void* saved, size_t saved_bytes, void* ws,
                    size_t ws_bytes, void* stream) {
  ScanSize c;
  gdn_status st = check_scan(p, false, &c);
  if (st != GDN_OK) return st;
  st = check_tensors({{u, c.values, 16, true}, {dt, c.values, 16, true}, {A, c.a, 16, true}, {Bm, c.bc, 16, true},
                      {Cm, c.bc, 16, true}, {Dskip, c.chan, 16, false}, {z, c.values, 16, false},
                      {dt_bias, c.chan, 16, false}, {h0, c.state, 16, false}},
                     {{y, c.values, 16, true}, {h_final, c.state, 16, false}, {saved, saved_bytes, 16, false},
                      {ws, ws_bytes, 16, false}});
  if (st != GDN_OK) return st;
  const size_t need = c.seg_end + c.seg_sum;
  if (need && (!ws || ws_bytes < need)) return GDN_ERR_WORKSPACE;
  if (save && c.saved && (!saved || saved_bytes < c.saved)) return GDN_ERR_WORKSPACE;
  if (p->num_seqs == 0) return GDN_OK;
  gdn::ScanParams sp = scan_params(p, c, u, dt, A, Bm, Cm, Dskip, z, dt_bias);
  sp.h0 = h0; sp.y = y; sp.h_final = h_final;
  sp.saved = save ? static_cast<float*>(saved) : nullptr;
  set_segments(&sp, c, ws);
  return hip_status(gdn::launch_scan_fwd(sp, p->N, c.io == 2, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

gdn_status gdn_step(const gdn_problem* p, const void* q, const void* k, const void* v, const float* g,
                    const float* beta, float* S, void* o, void* stream) {
  return step(p, q, k, v, g, beta, S, o, stream, false);
}

gdn_status gdn_kda_step(const gdn_problem* p, const void* q, const void* k, const void* v, const float* g,
                        const float* beta, float* S, void* o, void* stream) {
  return step(p, q, k, v, g, beta, S, o, stream, true);
}

gdn_status gdn_conv_fwd(const gdn_conv_problem* p, const void* x, const float* weight, const float* bias,
                        const void* state0, void* y, void* state_final, void* stream) {
  ConvSize c;
  gdn_status st = check_conv(p, &c);
  if (st != GDN_OK) return st;
  st = check_tensors({{x, c.values, 16, true}, {weight, c.weight, 16, true}, {bias, c.bias, 16, false},
                      {state0, c.state, 16, false}},
                     {{y, c.values, 16, true}, {state_final, c.state, 16, false}});
  if (st != GDN_OK || p->num_seqs == 0) return st;
  gdn::ConvParams cp = conv_params(p, c, x, weight, bias);
  cp.state0 = state0; cp.y = y; cp.state_final = state_final;
  return hip_status(gdn::launch_conv_fwd(cp, p->W, c.io == 2, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_conv_workspace_size(const gdn_conv_problem* p, size_t* bytes) {
  if (!bytes) return GDN_ERR_NULL;
  ConvSize c;
  const gdn_status st = check_conv(p, &c);
  if (st != GDN_OK) return st;
  *bytes = c.ws;
  return GDN_OK;
}

gdn_status gdn_conv_bwd(const gdn_conv_problem* p, const void* x, const float* weight, const float* bias,
                        const void* state0, const void* dy, const void* dstate_final, void* dx, float* dweight,
                        float* dbias, void* dstate0, void* ws, size_t ws_bytes, void* stream) {
  ConvSize c;
  gdn_status st = check_conv(p, &c);
  if (st != GDN_OK) return st;
  st = check_tensors({{x, c.values, 16, true}, {weight, c.weight, 16, true}, {bias, c.bias, 16, false},
                      {state0, c.state, 16, false}, {dy, c.values, 16, true}, {dstate_final, c.state, 16, false}},
                     {{dx, c.values, 16, true}, {dweight, c.weight, 16, true}, {dbias, c.bias, 16, false},
                      {dstate0, c.state, 16, false}, {ws, ws_bytes, 16, false}});
  if (st != GDN_OK) return st;
  if (c.ws && (!ws || ws_bytes < c.ws)) return GDN_ERR_WORKSPACE;
  gdn::ConvParams cp = conv_params(p, c, x, weight, bias);
  cp.state0 = state0; cp.dy = dy; cp.dstate_final = dstate_final;
  cp.dx = dx; cp.dweight = dweight; cp.dbias = dbias; cp.dstate0 = dstate0;
  cp.ws = static_cast<float*>(ws);
  return hip_status(gdn::launch_conv_bwd(cp, p->W, c.io == 2, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_conv_step(const gdn_conv_problem* p, const void* x, const float* weight, const float* bias,
                         void* state, void* y, void* stream) {
  ConvSize c;
  gdn_status st = check_conv(p, &c);
  if (st != GDN_OK) return st;
  if (p->T != 1 || p->cu_seqlens_host) return GDN_ERR_SHAPE;
  st = check_tensors({{x, c.values, 16, true}, {weight, c.weight, 16, true}, {bias, c.bias, 16, false}},
                     {{state, c.state, 16, true}, {y, c.values, 16, true}});
  if (st != GDN_OK || p->B == 0) return st;
  gdn::ConvParams cp = conv_params(p, c, x, weight, bias);
  cp.state_final = state; cp.y = y;
  return hip_status(gdn::launch_conv_step(cp, p->W, c.io == 2, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_scan_workspace_size(const gdn_scan_problem* p, int32_t pass, size_t* bytes) {
  if (!bytes) return GDN_ERR_NULL;
  if (pass != GDN_SCAN_FWD && pass != GDN_SCAN_SAVED && pass != GDN_SCAN_BWD) return GDN_ERR_UNSUPPORTED;
  ScanSize c;
  const gdn_status st = check_scan(p, pass == GDN_SCAN_BWD, &c);
  if (st != GDN_OK) return st;
  const size_t segments = c.seg_end + c.seg_sum;
  *bytes = pass == GDN_SCAN_SAVED ? c.saved : pass == GDN_SCAN_FWD ? segments : segments + c.part_bc + c.part_a;
  return GDN_OK;
}

gdn_status gdn_scan_fwd(const gdn_scan_problem* p, const void* u, const void* dt, const float* A, const void* Bm,
                        const void* Cm, const float* Dskip, const void* z, const float* dt_bias, const float* h0,
                        void* y, float* h_final, void* ws, size_t ws_bytes, void* stream) {
  return scan_fwd(p, u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, y, h_final, false, nullptr, 0, ws, ws_bytes, stream);
}

gdn_status gdn_scan_fwd_save(const gdn_scan_problem* p, const void* u, const void* dt, const float* A,
                             const void* Bm, const void* Cm, const float* Dskip, const void* z,
                             const float* dt_bias, const float* h0, void* y, float* h_final, void* saved,
                             size_t saved_bytes, void* ws, size_t ws_bytes, void* stream) {
  return scan_fwd(p, u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, y, h_final, true, saved, saved_bytes, ws, ws_bytes,
                  stream);
}

gdn_status gdn_scan_bwd_saved(const gdn_scan_problem* p, const void* u, const void* dt, const float* A,
                              const void* Bm, const void* Cm, const float* Dskip, const void* z,
                              const float* dt_bias, const void* dy, const float* dh_final, const void* saved,
                              size_t saved_bytes, void* du, void* ddt, float* dA, void* dBm, void* dCm,
                              float* dDskip, void* dz, float* ddt_bias, float* dh0, void* ws, size_t ws_bytes,
                              void* stream) {
  ScanSize c;
  gdn_status st = check_scan(p, true, &c);
  if (st != GDN_OK) return st;
  if (dz && !z) return GDN_ERR_NULL;
  st = check_tensors({{u, c.values, 16, true}, {dt, c.values, 16, true}, {A, c.a, 16, true}, {Bm, c.bc, 16, true},
                      {Cm, c.bc, 16, true}, {Dskip, c.chan, 16, false}, {z, c.values, 16, false},
                      {dt_bias, c.chan, 16, false}, {dy, c.values, 16, true}, {dh_final, c.state, 16, false},
                      {saved, saved_bytes, 16, false}},
                     {{du, c.values, 16, true}, {ddt, c.values, 16, true}, {dA, c.a, 16, true},
                      {dBm, c.bc, 16, true}, {dCm, c.bc, 16, true}, {dDskip, c.chan, 16, false},
                      {dz, c.values, 16, false}, {ddt_bias, c.chan, 16, false}, {dh0, c.state, 16, false},
                      {ws, ws_bytes, 16, false}});
  if (st != GDN_OK) return st;
  const size_t segments = c.seg_end + c.seg_sum, need = segments + c.part_bc + c.part_a;
  if (need && (!ws || ws_bytes < need)) return GDN_ERR_WORKSPACE;
  if (c.saved && (!saved || saved_bytes < c.saved)) return GDN_ERR_WORKSPACE;
  gdn::ScanParams sp = scan_params(p, c, u, dt, A, Bm, Cm, Dskip, z, dt_bias);
  sp.saved = const_cast<float*>(static_cast<const float*>(saved));
  sp.dy = dy; sp.dh_final = dh_final;
  sp.du = du; sp.ddt = ddt; sp.dA = dA; sp.dBm = dBm; sp.dCm = dCm; sp.dDskip = dDskip; sp.dz = dz;
  sp.ddt_bias = ddt_bias; sp.dh0 = dh0;
  set_segments(&sp, c, ws);
  if (need) {
    sp.part_bc = reinterpret_cast<float*>(static_cast<char*>(ws) + segments);
    sp.part_a = reinterpret_cast<float*>(static_cast<char*>(ws) + segments + c.part_bc);
  }
  return hip_status(gdn::launch_scan_bwd(sp, p->N, c.io == 2, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_scan_step(const gdn_scan_problem* p, const void* u, const void* dt, const float* A, const void* Bm,
                         const void* Cm, const float* Dskip, const void* z, const float* dt_bias, float* h,
                         void* y, void* stream) {
  ScanSize c;
  gdn_status st = check_scan(p, false, &c);
  if (st != GDN_OK) return st;
  if (p->T != 1 || p->cu_seqlens_host) return GDN_ERR_SHAPE;
  st = check_tensors({{u, c.values, 16, true}, {dt, c.values, 16, true}, {A, c.a, 16, true}, {Bm, c.bc, 16, true},
                      {Cm, c.bc, 16, true}, {Dskip, c.chan, 16, false}, {z, c.values, 16, false},
                      {dt_bias, c.chan, 16, false}},
                     {{h, c.state, 16, true}, {y, c.values, 16, true}});
  if (st != GDN_OK || p->B == 0) return st;
  gdn::ScanParams sp = scan_params(p, c, u, dt, A, Bm, Cm, Dskip, z, dt_bias);
  sp.h_final = h; sp.y = y;
  return hip_status(gdn::launch_scan_step(sp, p->N, c.io == 2, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
