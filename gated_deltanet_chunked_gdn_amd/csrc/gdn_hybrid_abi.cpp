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

}  // extern "C"
