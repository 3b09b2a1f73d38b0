// C ABI of the operators that hybrid models put next to the delta rule (gdn_glr_*,
// gdn_rope_*, gdn_swa_*): argument validation, workspace sizing and dispatch.  Every check
// runs on the host before the first launch (see include/gdn.h).
#include "gdn.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gdn_abi_check.h"
#include "gdn_hybrid.h"

using gdn::check::check_seqs;
using gdn::check::check_tensors;
using gdn::check::hip_status;
using gdn::check::up256;

namespace {

// ---------------------------------------------------------------------------- recurrence

struct GlrSize {
  size_t io = 0, values = 0, chan = 0, state = 0, saved = 0, seg = 0, part = 0;
  int64_t rows = 0, seg_len = 1;
  int32_t segs = 1, waves = 1;
};

// Tokens of a wave: 64 lanes over the lanes of a row (eight in the forward, of four channels;
// sixteen in the backward, of two), eight tokens each.
constexpr int64_t kFwdWave = 64, kBwdWave = 32;

gdn_status check_glr(const gdn_glr_problem* p, bool bwd, GlrSize* c) {
  if (!p) return GDN_ERR_NULL;
  if (p->io_dtype != GDN_FP32 && p->io_dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (p->B < 0 || p->T < 0 || p->C <= 0 || p->num_seqs < 0) return GDN_ERR_SHAPE;
  if (p->C % 8 != 0 || p->C > 1 << 20 || !(p->c >= 0.f)) return GDN_ERR_UNSUPPORTED;
  int64_t max_len = 0;
  const gdn_status st = check_seqs(p, &max_len);
  if (st != GDN_OK) return st;
  c->io = p->io_dtype == GDN_BF16 ? 2 : 4;
  c->rows = static_cast<int64_t>(p->B) * p->T;
  if (c->rows > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  c->values = static_cast<size_t>(c->rows) * p->C * c->io;
  c->chan = static_cast<size_t>(p->C) * 4;
  c->state = static_cast<size_t>(p->num_seqs) * c->chan;
  c->saved = static_cast<size_t>(gdn::glr_slots(c->rows, p->num_seqs)) * c->chan;
  // A tile as long as the longest sequence needs, up to eight waves.
  const int64_t wave = bwd ? kBwdWave : kFwdWave;
  c->waves = max_len <= wave ? 1 : max_len <= 4 * wave ? 4 : 8;
  // Segments where the channels leave CUs idle, of two tiles at least.
  const int64_t tile = wave * c->waves, tiles = gdn::glr_tiles(p->C);
  const int64_t groups = std::max<int64_t>(1, (c->rows + std::max<int64_t>(max_len, 1) - 1) / std::max<int64_t>(max_len, 1)) * tiles;
  const int64_t segs = std::max<int64_t>(1, std::min<int64_t>((256 + groups - 1) / groups, max_len / (2 * tile)));
  c->seg_len = std::max<int64_t>(((max_len + segs - 1) / segs + tile - 1) / tile * tile, tile);
  c->segs = static_cast<int32_t>(std::max<int64_t>(1, (max_len + c->seg_len - 1) / c->seg_len));
  const size_t parts = static_cast<size_t>(gdn::glr_parts(c->rows, p->num_seqs, c->seg_len));
  c->seg = c->segs > 1 ? up256(parts * 2 * c->chan) : 0;
  c->part = bwd ? parts * c->chan : 0;
  // a launch counts its threads in 32 bits; the step has fewer than any other
  if (static_cast<int64_t>((tiles + 7) / 8 * 8) * p->num_seqs * c->segs * 64 * c->waves >= INT64_C(1) << 32) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

gdn::GlrParams glr_params(const gdn_glr_problem* p, const GlrSize& c, const void* x, const void* r, const void* i,
                          const float* lam, const void* z) {
  gdn::GlrParams gp{};
  gp.x = x; gp.r = r; gp.i = i; gp.lam = lam; gp.z = z;
  gp.seq = gdn::SeqInfo{p->cu_seqlens_dev, p->T};
  gp.rows = c.rows; gp.N = p->num_seqs; gp.C = p->C;
  gp.segs = c.segs; gp.seg_len = c.seg_len; gp.waves = c.waves;
  gp.c = p->c;
  return gp;
}

gdn_status glr_fwd(const gdn_glr_problem* p, const void* x, const void* r, const void* i, const float* lam, const void* z,
                   const float* h0, void* y, float* h_final, bool save, void* saved, size_t saved_bytes, void* ws,
                   size_t ws_bytes, void* stream) {
  GlrSize c;
  gdn_status st = check_glr(p, false, &c);
  if (st != GDN_OK) return st;
  st = check_tensors({{x, c.values, 16, true}, {r, c.values, 16, true}, {i, c.values, 16, true}, {lam, c.chan, 16, true},
                      {z, c.values, 16, false}, {h0, c.state, 16, false}},
                     {{y, c.values, 16, true}, {h_final, c.state, 16, false}, {saved, saved_bytes, 16, false},
                      {ws, ws_bytes, 16, false}});
  if (st != GDN_OK) return st;
  if (c.seg && (!ws || ws_bytes < c.seg)) return GDN_ERR_WORKSPACE;
  if (save && (!saved || saved_bytes < c.saved)) return GDN_ERR_WORKSPACE;
  if (p->num_seqs == 0) return GDN_OK;
  gdn::GlrParams gp = glr_params(p, c, x, r, i, lam, z);
  gp.h0 = h0; gp.y = y; gp.h_final = h_final;
  gp.saved = save ? static_cast<float*>(saved) : nullptr;
  gp.seg = static_cast<float*>(ws);
  return hip_status(gdn::launch_glr_fwd(gp, c.io == 2, static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------------------- norm and rotation

struct RopeSize {
  size_t io = 0, qin = 0, kin = 0, q = 0, k = 0, freq = 0, pos = 0, weight = 0, ws = 0;
  int64_t tokens = 0, q_stride = 0, k_stride = 0;
};

// Bytes from the first to the last value of `rows` rows of `row` values, `stride` apart.
size_t extent(int64_t rows, int64_t stride, int64_t row, size_t io) {
  return rows ? static_cast<size_t>((rows - 1) * stride + row) * io : 0;
}

// A row stride in values (0: the row itself): whole 16 bytes, rows that do not overlap.
gdn_status check_stride(int64_t given, int64_t row, size_t io, int64_t* stride) {
  *stride = given ? given : row;
  if (*stride < row) return GDN_ERR_SHAPE;
  // 2^31 rows of 2^31 values of 4 bytes would pass 64 bits
  if (*stride > INT64_C(1) << 28) return GDN_ERR_UNSUPPORTED;
  return *stride * static_cast<int64_t>(io) % 16 ? GDN_ERR_ALIGN : GDN_OK;
}

gdn_status check_rope(const gdn_rope_problem* p, RopeSize* c) {
  if (!p) return GDN_ERR_NULL;
  if (p->io_dtype != GDN_FP32 && p->io_dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (p->B < 0 || p->T < 0 || p->Hq <= 0 || p->Hk <= 0 || p->D <= 0 || p->R < 0 || p->R > p->D) return GDN_ERR_SHAPE;
  if ((p->D != 64 && p->D != 128 && p->D != 256) || p->R % 16 != 0 || p->Hq > 4096 || p->Hk > 4096) return GDN_ERR_UNSUPPORTED;
  if (p->norm != GDN_ROPE_NONE && p->norm != GDN_ROPE_RMS && p->norm != GDN_ROPE_L2) return GDN_ERR_UNSUPPORTED;
  c->io = p->io_dtype == GDN_BF16 ? 2 : 4;
  c->tokens = static_cast<int64_t>(p->B) * p->T;
  if (c->tokens > INT32_MAX || c->tokens * (p->Hq + p->Hk) > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  // 256 threads for every four tokens and more (one below 4096), counted in 32 bits
  if (c->tokens / gdn::kRopeMost >= INT64_C(1) << 24) return GDN_ERR_UNSUPPORTED;
  const int64_t qrow = static_cast<int64_t>(p->Hq) * p->D, krow = static_cast<int64_t>(p->Hk) * p->D;
  gdn_status st = check_stride(p->q_stride, qrow, c->io, &c->q_stride);
  if (st == GDN_OK) st = check_stride(p->k_stride, krow, c->io, &c->k_stride);
  if (st != GDN_OK) return st;
  c->qin = extent(c->tokens, c->q_stride, qrow, c->io);
  c->kin = extent(c->tokens, c->k_stride, krow, c->io);
  c->q = static_cast<size_t>(c->tokens) * qrow * c->io;
  c->k = static_cast<size_t>(c->tokens) * krow * c->io;
  c->freq = static_cast<size_t>(p->R) / 2 * 4;
  c->pos = static_cast<size_t>(c->tokens) * 4;
  c->weight = static_cast<size_t>(p->D) * 4;
  c->ws = static_cast<size_t>(gdn::rope_bwd_groups(c->tokens)) * 2 * c->weight;
  return GDN_OK;
}

gdn::RopeParams rope_params(const gdn_rope_problem* p, const RopeSize& c, const void* q, const void* k, const float* inv_freq,
                            const int32_t* positions, const float* wq, const float* wk) {
  gdn::RopeParams rp{};
  rp.q = q; rp.k = k; rp.inv_freq = inv_freq; rp.pos = positions; rp.wq = wq; rp.wk = wk;
  rp.q_stride = c.q_stride; rp.k_stride = c.k_stride; rp.tokens = c.tokens;
  rp.T = p->T; rp.Hq = p->Hq; rp.Hk = p->Hk; rp.R = p->R; rp.norm = p->norm; rp.eps = p->eps;
  rp.per_group = gdn::rope_tokens(c.tokens);
  return rp;
}

}  // namespace

extern "C" {

gdn_status gdn_glr_workspace_size(const gdn_glr_problem* p, int32_t pass, size_t* bytes) {
  if (!bytes) return GDN_ERR_NULL;
  if (pass != GDN_GLR_FWD && pass != GDN_GLR_SAVED && pass != GDN_GLR_BWD) return GDN_ERR_UNSUPPORTED;
  GlrSize c;
  const gdn_status st = check_glr(p, pass == GDN_GLR_BWD, &c);
  if (st != GDN_OK) return st;
  *bytes = pass == GDN_GLR_SAVED ? c.saved : c.seg + c.part;
  return GDN_OK;
}

gdn_status gdn_glr_fwd(const gdn_glr_problem* p, const void* x, const void* r, const void* i, const float* lam,
                       const void* z, const float* h0, void* y, float* h_final, void* ws, size_t ws_bytes, void* stream) {
  return glr_fwd(p, x, r, i, lam, z, h0, y, h_final, false, nullptr, 0, ws, ws_bytes, stream);
}

gdn_status gdn_glr_fwd_save(const gdn_glr_problem* p, const void* x, const void* r, const void* i, const float* lam,
                            const void* z, const float* h0, void* y, float* h_final, void* saved, size_t saved_bytes,
                            void* ws, size_t ws_bytes, void* stream) {
  return glr_fwd(p, x, r, i, lam, z, h0, y, h_final, true, saved, saved_bytes, ws, ws_bytes, stream);
}

gdn_status gdn_glr_bwd_saved(const gdn_glr_problem* p, const void* x, const void* r, const void* i, const float* lam,
                             const void* z, const void* dy, const float* dh_final, const void* saved, size_t saved_bytes,
                             void* dx, void* dr, void* di, float* dlam, void* dz, float* dh0, void* ws, size_t ws_bytes,
                             void* stream) {
  GlrSize c;
  gdn_status st = check_glr(p, true, &c);
  if (st != GDN_OK) return st;
  if (dz && !z) return GDN_ERR_NULL;
  st = check_tensors({{x, c.values, 16, true}, {r, c.values, 16, true}, {i, c.values, 16, true}, {lam, c.chan, 16, true},
                      {z, c.values, 16, false}, {dy, c.values, 16, true}, {dh_final, c.state, 16, false},
                      {saved, saved_bytes, 16, false}},
                     {{dx, c.values, 16, true}, {dr, c.values, 16, true}, {di, c.values, 16, true}, {dlam, c.chan, 16, true},
                      {dz, c.values, 16, false}, {dh0, c.state, 16, false}, {ws, ws_bytes, 16, false}});
  if (st != GDN_OK) return st;
  if (c.seg + c.part && (!ws || ws_bytes < c.seg + c.part)) return GDN_ERR_WORKSPACE;
  if (!saved || saved_bytes < c.saved) return GDN_ERR_WORKSPACE;
  gdn::GlrParams gp = glr_params(p, c, x, r, i, lam, z);
  gp.saved = const_cast<float*>(static_cast<const float*>(saved));
  gp.dy = dy; gp.dh_final = dh_final;
  gp.dx = dx; gp.dr = dr; gp.di = di; gp.dlam = dlam; gp.dz = dz; gp.dh0 = dh0;
  gp.seg = static_cast<float*>(ws);
  gp.part_lam = reinterpret_cast<float*>(static_cast<char*>(ws) + c.seg);
  return hip_status(gdn::launch_glr_bwd(gp, c.io == 2, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_glr_step(const gdn_glr_problem* p, const void* x, const void* r, const void* i, const float* lam,
                        const void* z, float* h, void* y, void* stream) {
  GlrSize c;
  gdn_status st = check_glr(p, false, &c);
  if (st != GDN_OK) return st;
  if (p->T != 1 || p->cu_seqlens_host) return GDN_ERR_SHAPE;
  st = check_tensors({{x, c.values, 16, true}, {r, c.values, 16, true}, {i, c.values, 16, true}, {lam, c.chan, 16, true},
                      {z, c.values, 16, false}},
                     {{h, c.state, 16, true}, {y, c.values, 16, true}});
  if (st != GDN_OK || p->B == 0) return st;
  gdn::GlrParams gp = glr_params(p, c, x, r, i, lam, z);
  gp.h_final = h; gp.y = y;
  return hip_status(gdn::launch_glr_step(gp, c.io == 2, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_rope_fwd(const gdn_rope_problem* p, const void* q, const void* k, const float* inv_freq,
                        const int32_t* positions, const float* wq, const float* wk, void* q_out, void* k_out, void* stream) {
  RopeSize c;
  gdn_status st = check_rope(p, &c);
  if (st != GDN_OK) return st;
  if ((wq || wk) && p->norm != GDN_ROPE_RMS) return GDN_ERR_UNSUPPORTED;
  st = check_tensors({{q, c.qin, 16, true}, {k, c.kin, 16, true}, {inv_freq, c.freq, 4, true}, {positions, c.pos, 4, false},
                      {wq, c.weight, 16, false}, {wk, c.weight, 16, false}},
                     {{q_out, c.q, 16, true}, {k_out, c.k, 16, true}});
  if (st != GDN_OK || c.tokens == 0) return st;
  gdn::RopeParams rp = rope_params(p, c, q, k, inv_freq, positions, wq, wk);
  rp.q_out = q_out; rp.k_out = k_out;
  rp.groups = static_cast<int32_t>((c.tokens + rp.per_group - 1) / rp.per_group);
  return hip_status(gdn::launch_rope_fwd(rp, p->D, c.io == 2, p->interleaved != 0, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_rope_workspace_size(const gdn_rope_problem* p, size_t* bytes) {
  if (!bytes) return GDN_ERR_NULL;
  RopeSize c;
  const gdn_status st = check_rope(p, &c);
  if (st != GDN_OK) return st;
  *bytes = c.ws;
  return GDN_OK;
}

gdn_status gdn_rope_bwd(const gdn_rope_problem* p, const void* q, const void* k, const float* inv_freq,
                        const int32_t* positions, const float* wq, const float* wk, const void* dq_out, const void* dk_out,
                        void* dq, void* dk, float* dwq, float* dwk, void* ws, size_t ws_bytes, void* stream) {
  RopeSize c;
  gdn_status st = check_rope(p, &c);
  if (st != GDN_OK) return st;
  if ((wq || wk || dwq || dwk) && p->norm != GDN_ROPE_RMS) return GDN_ERR_UNSUPPORTED;
  st = check_tensors({{q, c.qin, 16, true}, {k, c.kin, 16, true}, {inv_freq, c.freq, 4, true}, {positions, c.pos, 4, false},
                      {wq, c.weight, 16, false}, {wk, c.weight, 16, false}, {dq_out, c.q, 16, true}, {dk_out, c.k, 16, true}},
                     {{dq, c.q, 16, true}, {dk, c.k, 16, true}, {dwq, c.weight, 16, false}, {dwk, c.weight, 16, false},
                      {ws, ws_bytes, 16, false}});
  if (st != GDN_OK) return st;
  if ((dwq || dwk) && c.ws && (!ws || ws_bytes < c.ws)) return GDN_ERR_WORKSPACE;
  if (c.tokens == 0 && !dwq && !dwk) return GDN_OK;
  gdn::RopeParams rp = rope_params(p, c, q, k, inv_freq, positions, wq, wk);
  rp.q_out = dq; rp.k_out = dk; rp.dq_out = dq_out; rp.dk_out = dk_out; rp.dwq = dwq; rp.dwk = dwk;
  rp.part = static_cast<float*>(ws);
  rp.groups = static_cast<int32_t>(gdn::rope_bwd_groups(c.tokens));
  return hip_status(gdn::launch_rope_bwd(rp, p->D, c.io == 2, p->interleaved != 0, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
