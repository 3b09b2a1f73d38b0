// C ABI of the operators that hybrid models put next to the delta rule (gdn_glr_*,
// gdn_rope_*, gdn_swa_*): argument validation, workspace sizing and dispatch.  Every check
// runs on the host before the first launch (see include/gdn.h).
#include "gdn.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
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
  size_t io = 0, values = 0, chan = 0, state = 0, saved = 0;
  size_t whole = 0, end = 0, part = 0;  // words of the segments and groups, partial sums
  int64_t rows = 0, slots = 0;
  int32_t chained = 0;
  // the counter, then the words: what is cleared before a launch
  size_t chain() const { return chained ? 256 + whole + end : 0; }
};

gdn_status check_glr(const gdn_glr_problem* p, bool bwd, GlrSize* c) {
  if (!p) return GDN_ERR_NULL;
  if (p->io_dtype != GDN_FP32 && p->io_dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (p->B < 0 || p->T < 0 || p->C <= 0 || p->num_seqs < 0) return GDN_ERR_SHAPE;
  if (p->C % 8 != 0 || p->C > 1 << 20 || !(p->c >= 0.f) || !std::isfinite(p->c)) return GDN_ERR_UNSUPPORTED;
  int64_t max_len = 0;
  const gdn_status st = check_seqs(p, &max_len);
  if (st != GDN_OK) return st;
  c->io = p->io_dtype == GDN_BF16 ? 2 : 4;
  c->rows = static_cast<int64_t>(p->B) * p->T;
  if (c->rows > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  c->values = static_cast<size_t>(c->rows) * p->C * c->io;
  c->chan = static_cast<size_t>(p->C) * 4;
  c->state = static_cast<size_t>(p->num_seqs) * c->chan;
  c->saved = static_cast<size_t>(gdn::glr_slots(c->rows, p->num_seqs, gdn::kGlrRun)) * c->chan;
  const int64_t seg = gdn::glr_seg(bwd);
  // dense sequences have the slots that their segments need (one, of no tokens, where T is 0)
  const auto slots = [p, c](int64_t len) {
    return p->cu_seqlens_host ? gdn::glr_slots(c->rows, p->num_seqs, len) : p->B * std::max<int64_t>(1, (p->T + len - 1) / len);
  };
  c->slots = slots(seg);
  c->chained = max_len > seg;
  const size_t words = static_cast<size_t>(gdn::glr_tiles(p->C)) * gdn::kGlrTile * 8;
  c->whole = static_cast<size_t>(c->slots) * words;
  c->end = static_cast<size_t>(gdn::glr_slots(c->rows, p->num_seqs, seg * gdn::kGlrGroup)) * words;
  c->part = bwd ? static_cast<size_t>(c->slots) * c->chan : 0;
  // workgroups of 256 threads, counted in 32 bits: segments of the longer of the two
  // directions' segments or shorter, so that what the forward takes the backward takes too
  const int64_t most = slots(gdn::glr_seg(true));
  if (most * gdn::glr_tiles(p->C) >= 1 << 24) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

gdn::GlrParams glr_params(const gdn_glr_problem* p, const GlrSize& c, const void* x, const void* r, const void* i,
                          const float* lam, const void* z, void* ws) {
  gdn::GlrParams gp{};
  gp.x = x; gp.r = r; gp.i = i; gp.lam = lam; gp.z = z;
  gp.seq = gdn::SeqInfo{p->cu_seqlens_dev, p->T};
  gp.rows = c.rows; gp.N = p->num_seqs; gp.C = p->C;
  gp.words = gdn::glr_tiles(p->C) * gdn::kGlrTile;
  gp.slots = c.slots; gp.chained = c.chained;
  gp.c = p->c;
  if (c.chained) {
    char* const at = static_cast<char*>(ws);
    gp.chain = reinterpret_cast<uint64_t*>(at);
    gp.whole = reinterpret_cast<uint64_t*>(at + 256);
    gp.end = reinterpret_cast<uint64_t*>(at + 256 + c.whole);
  }
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
  if (c.chained && (!ws || ws_bytes < c.chain())) return GDN_ERR_WORKSPACE;
  if (save && c.saved && (!saved || saved_bytes < c.saved)) return GDN_ERR_WORKSPACE;
  if (p->num_seqs == 0) return GDN_OK;
  gdn::GlrParams gp = glr_params(p, c, x, r, i, lam, z, ws);
  gp.h0 = h0; gp.y = y; gp.h_final = h_final;
  gp.saved = save ? static_cast<float*>(saved) : nullptr;
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
  // The attention's kernels address up to 128 rows from one of them in 32 bits.  The rotation and
  // the cache's calls go by 64 bits; they have the same limit, so that what one of the calls takes
  // the others take.
  if (*stride > INT64_C(1) << 21) return GDN_ERR_UNSUPPORTED;
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
  c->ws = static_cast<size_t>(gdn::rope_groups(c->tokens)) * 2 * c->weight;
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

// ---------------------------------------------------------------------------- window attention

struct SwaSize {
  size_t io = 0, qin = 0, kin = 0, vin = 0, q = 0, k = 0, lse = 0, cache = 0, lens = 0;
  size_t delta = 0, win = 0, far = 0, step = 0;
  int64_t rows = 0, q_stride = 0, k_stride = 0, v_stride = 0;
  int32_t W = 0, S = 0, few = 0, few_keys = 0, run_far = 256, splits = 1, run = 0;
};

gdn_status check_swa(const gdn_swa_problem* p, SwaSize* c) {
  if (!p) return GDN_ERR_NULL;
  if (p->io_dtype != GDN_FP32 && p->io_dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (p->B < 0 || p->T < 0 || p->Hq <= 0 || p->Hk <= 0 || p->D <= 0 || p->num_seqs < 0 || p->Hq % p->Hk != 0 || p->window <= 0 || p->sinks < 0)
    return GDN_ERR_SHAPE;
  if ((p->D != 64 && p->D != 128) || p->Hq > 4096 || p->sinks > 1024 || !std::isfinite(p->scale)) return GDN_ERR_UNSUPPORTED;
  int64_t max_len = 0;
  gdn_status st = check_seqs(p, &max_len);
  if (st != GDN_OK) return st;
  c->io = p->io_dtype == GDN_BF16 ? 2 : 4;
  c->rows = static_cast<int64_t>(p->B) * p->T;
  if (c->rows > 1 << 30) return GDN_ERR_UNSUPPORTED;
  const int64_t qrow = static_cast<int64_t>(p->Hq) * p->D, krow = static_cast<int64_t>(p->Hk) * p->D;
  st = check_stride(p->q_stride, qrow, c->io, &c->q_stride);
  if (st == GDN_OK) st = check_stride(p->k_stride, krow, c->io, &c->k_stride);
  if (st == GDN_OK) st = check_stride(p->v_stride, krow, c->io, &c->v_stride);
  if (st != GDN_OK) return st;
  // a window as long as every sequence leaves nothing behind it
  c->W = static_cast<int32_t>(std::min<int64_t>(p->window, std::max<int64_t>(max_len, 1)));
  c->S = c->W >= max_len ? 0 : static_cast<int32_t>(std::min<int64_t>(p->sinks, max_len));
  c->qin = extent(c->rows, c->q_stride, qrow, c->io);
  c->kin = extent(c->rows, c->k_stride, krow, c->io);
  c->vin = extent(c->rows, c->v_stride, krow, c->io);
  c->q = static_cast<size_t>(c->rows) * qrow * c->io;
  c->k = static_cast<size_t>(c->rows) * krow * c->io;
  c->lse = static_cast<size_t>(c->rows) * p->Hq * 4;
  c->delta = up256(c->lse);
  const size_t first = static_cast<size_t>(p->Hk) * c->S * 2 * p->D * 4;
  c->win = up256(p->num_seqs * first);
  // Runs of 256 queries for the first tokens' sums, or of a tile of them where those leave most
  // CUs without work.  Training steps, us, by runs of 64, 128 and 256 queries: 10 runs of 256 (five
  // sequences, 1501 tokens, 2 key heads, fp32, D = 64) 85, 90, 104; 64 (4096 tokens, 4 key heads of
  // 128) bf16 211, 202, 206, fp32 989, 991, 1015; 512 (16384 tokens, 8 key heads of 128) bf16 598,
  // 544, 521, fp32 3927, 3884, 3869.
  const int64_t far = c->rows / 256 * p->Hk * ((c->S + 15) / 16);
  c->run_far = far >= 128 ? 256 : c->io == 2 ? 128 : 64;
  c->far = static_cast<size_t>(gdn::swa_far_slots(c->rows, p->num_seqs, c->run_far)) * first;
  // Blocks of half as many queries, or of a quarter as many keys, where whole ones leave CUs
  // without work (packed sequences of other lengths count as so many of the rows).  Training steps
  // over one sequence, window 512, us, halves | whole, by tokens and heads of queries / of keys:
  //   blocks of queries            bf16, D = 128   fp32, D = 128   bf16, D = 64   fp32, D = 64
  //   256  (2048, 16 / 4)              98 | 104       472 | 461        69 | 75       231 | 244
  //   384  (4096, 12 / 4)             151 | 150       712 | 815        74 | 82       308 | 365
  //   512  (4096, 16 / 4)             184 | 174       941 | 915        91 | 93       396 | 407
  //   1024 (8192, 16 / 8)             262 | 234      1892 | 1834      148 | 149      783 | 807
  // and quarters | whole:
  //   blocks of keys               bf16, D = 128   fp32, D = 128   bf16, D = 64   fp32, D = 64
  //   128  (4096, 16 / 4)             174 | 216       915 | 1286       93 | 156      407 | 628
  //   256  (4096, 16 / 8)             179 | 144       923 | 919        94 | 101      411 | 435
  //   320  (4096, 20 / 10)            249 | 203      1285 | 1557      131 | 137      625 | 716
  //   512  (4096, 16 / 16)            209 | 135       950 | 936       102 | 85       422 | 417
  // (256 blocks fill the CUs once, 320 take a second turn.)  The bounds are those of bf16, for queries
  // of D = 128: fp32 at 384 blocks of queries or 320 of keys, and D = 64 from 384 blocks of queries
  // on, stand on the side that the table shows to be the slower one.
  const int64_t whole = c->rows / gdn::kSwaQueries;
  c->few = whole * p->Hq < 384;
  c->few_keys = whole * p->Hk < (p->D == 64 ? 320 : 256);
  return GDN_OK;
}

// The limit on the attention's workgroups, whose numbers are 32-bit: blocks of 32 rows (the launches'
// are as long or longer) of every sequence and query head, and what the first tokens add.
gdn_status check_swa_grid(const gdn_swa_problem* p, const SwaSize& c) {
  if (c.rows == 0) return GDN_OK;
  const auto blocks = [p](int64_t each) {
    const int32_t* const cu = p->cu_seqlens_host;
    if (!cu) return p->num_seqs * ((p->T + each - 1) / each);
    int64_t sum = 0;
    for (int32_t n = 0; n < p->num_seqs; ++n) sum += std::max<int64_t>(1, (cu[n + 1] - cu[n] + each - 1) / each);
    return sum;
  };
  const int64_t most = (1 << 24) - 1;
  const bool fits = blocks(32) * p->Hq <= most && blocks(c.run_far) * p->Hk * ((c.S + 15) / 16) <= most &&
                    static_cast<int64_t>(c.S) * p->Hk * p->num_seqs <= most;
  return fits ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

// What the cache adds: its slots, and the step's runs of them.
gdn_status check_cache(const gdn_swa_problem* p, SwaSize* c) {
  const gdn_status st = check_swa(p, c);
  if (st != GDN_OK) return st;
  const int64_t slots = static_cast<int64_t>(p->sinks) + p->window, row = static_cast<int64_t>(p->Hk) * p->D;
  if (slots > 1 << 30) return GDN_ERR_UNSUPPORTED;
  // threads of the filling: a piece of 16 bytes each; workgroups of the step
  const int64_t fill = (slots * (row * static_cast<int64_t>(c->io) / 16) + 255) / 256 * p->num_seqs;
  if (fill >= 1 << 24) return GDN_ERR_UNSUPPORTED;
  c->cache = static_cast<size_t>(p->num_seqs) * slots * row * c->io;
  c->lens = static_cast<size_t>(p->num_seqs) * 4;
  const int64_t groups = std::max<int64_t>(1, static_cast<int64_t>(p->num_seqs) * p->Hk * ((p->Hq / p->Hk + 15) / 16));
  // Whole where there is a workgroup a CU, else runs of at least 128 slots (32 a wave) that make
  // some 512 workgroups.  Aims of 256, 512 and 1024, us, 16 / 4 heads of 128: bf16, one sequence of
  // 30000 slots 21, 24, 32; eight 83, 74, 67; 16 of 4100 slots 35, 32, 30; 48 90, 82, 80; fp32 38,
  // 37, 46; 170, 131, 135; 63, 56, 62; 159, 172, 157.  64 of 4100 whole 97, as two runs 104.
  const int64_t splits = groups >= 256 ? 1 : std::min<int64_t>((512 + groups - 1) / groups, (slots + 127) / 128);
  c->run = static_cast<int32_t>(((slots + splits - 1) / splits + 127) / 128 * 128);
  c->splits = static_cast<int32_t>((slots + c->run - 1) / c->run);
  if (groups * c->splits >= 1 << 24) return GDN_ERR_UNSUPPORTED;
  c->step = c->splits > 1 ? static_cast<size_t>(c->splits) * p->num_seqs * p->Hq * (p->D + 2) * 4 : 0;
  return GDN_OK;
}

gdn::SwaParams swa_params(const gdn_swa_problem* p, const SwaSize& c, const void* q, const void* k, const void* v) {
  gdn::SwaParams sp{};
  sp.q = q; sp.k = k; sp.v = v;
  sp.q_stride = c.q_stride; sp.k_stride = c.k_stride; sp.v_stride = c.v_stride;
  sp.seq = gdn::SeqInfo{p->cu_seqlens_dev, p->T};
  sp.rows = c.rows; sp.N = p->num_seqs; sp.Hq = p->Hq; sp.Hk = p->Hk; sp.W = c.W; sp.S = c.S;
  sp.few = c.few; sp.few_keys = c.few_keys; sp.far = c.run_far;
  sp.scale = p->scale;
  return sp;
}

}  // namespace

extern "C" {

gdn_status gdn_glr_workspace_size(const gdn_glr_problem* p, int32_t pass, size_t* bytes) {
  if (!bytes) return GDN_ERR_NULL;
  if (pass != GDN_GLR_FWD && pass != GDN_GLR_SAVED && pass != GDN_GLR_BWD) return GDN_ERR_UNSUPPORTED;
  GlrSize c;
  const gdn_status st = check_glr(p, pass == GDN_GLR_BWD, &c);
  if (st != GDN_OK) return st;
  *bytes = pass == GDN_GLR_SAVED ? c.saved : c.chain() + c.part;
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
  const size_t need = c.chain() + c.part;
  if (need && (!ws || ws_bytes < need)) return GDN_ERR_WORKSPACE;
  if (c.saved && (!saved || saved_bytes < c.saved)) return GDN_ERR_WORKSPACE;
  gdn::GlrParams gp = glr_params(p, c, x, r, i, lam, z, ws);
  gp.saved = const_cast<float*>(static_cast<const float*>(saved));
  gp.dy = dy; gp.dh_final = dh_final;
  gp.dx = dx; gp.dr = dr; gp.di = di; gp.dlam = dlam; gp.dz = dz; gp.dh0 = dh0;
  gp.part_lam = reinterpret_cast<float*>(static_cast<char*>(ws) + c.chain());
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
  gdn::GlrParams gp = glr_params(p, c, x, r, i, lam, z, nullptr);
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
  rp.groups = static_cast<int32_t>(gdn::rope_groups(c.tokens));
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
  rp.groups = static_cast<int32_t>(gdn::rope_groups(c.tokens));
  return hip_status(gdn::launch_rope_bwd(rp, p->D, c.io == 2, p->interleaved != 0, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_swa_workspace_size(const gdn_swa_problem* p, int32_t pass, size_t* bytes) {
  if (!bytes) return GDN_ERR_NULL;
  if (pass != GDN_SWA_BWD && pass != GDN_SWA_STEP) return GDN_ERR_UNSUPPORTED;
  SwaSize c;
  gdn_status st = pass == GDN_SWA_BWD ? check_swa(p, &c) : check_cache(p, &c);
  if (st == GDN_OK) st = check_swa_grid(p, c);
  if (st != GDN_OK) return st;
  *bytes = pass == GDN_SWA_BWD ? c.delta + c.win + c.far : c.step;
  return GDN_OK;
}

gdn_status gdn_swa_fwd(const gdn_swa_problem* p, const void* q, const void* k, const void* v, void* o, float* lse, void* stream) {
  SwaSize c;
  gdn_status st = check_swa(p, &c);
  if (st == GDN_OK) st = check_swa_grid(p, c);
  if (st != GDN_OK) return st;
  st = check_tensors({{q, c.qin, 16, true}, {k, c.kin, 16, true}, {v, c.vin, 16, true}}, {{o, c.q, 16, true}, {lse, c.lse, 4, false}});
  if (st != GDN_OK || c.rows == 0) return st;
  gdn::SwaParams sp = swa_params(p, c, q, k, v);
  sp.o = o; sp.lse = lse;
  return hip_status(gdn::launch_swa_fwd(sp, p->D, c.io == 2, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_swa_bwd(const gdn_swa_problem* p, const void* q, const void* k, const void* v, const void* o, const float* lse,
                       const void* dout, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
  SwaSize c;
  gdn_status st = check_swa(p, &c);
  if (st == GDN_OK) st = check_swa_grid(p, c);
  if (st != GDN_OK) return st;
  st = check_tensors({{q, c.qin, 16, true}, {k, c.kin, 16, true}, {v, c.vin, 16, true}, {o, c.q, 16, true}, {lse, c.lse, 4, true},
                      {dout, c.q, 16, true}},
                     {{dq, c.q, 16, true}, {dk, c.k, 16, true}, {dv, c.k, 16, true}, {ws, ws_bytes, 16, false}});
  if (st != GDN_OK) return st;
  if (c.rows == 0) return GDN_OK;
  if (!ws || ws_bytes < c.delta + c.win + c.far) return GDN_ERR_WORKSPACE;
  gdn::SwaParams sp = swa_params(p, c, q, k, v);
  sp.o = const_cast<void*>(o); sp.lse = const_cast<float*>(lse); sp.dout = dout;
  sp.dq = dq; sp.dk = dk; sp.dv = dv;
  sp.delta = static_cast<float*>(ws);
  sp.first_win = reinterpret_cast<float*>(static_cast<char*>(ws) + c.delta);
  sp.first_far = reinterpret_cast<float*>(static_cast<char*>(ws) + c.delta + c.win);
  return hip_status(gdn::launch_swa_bwd(sp, p->D, c.io == 2, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_swa_fill(const gdn_swa_problem* p, const void* k, const void* v, void* kcache, void* vcache, void* stream) {
  SwaSize c;
  gdn_status st = check_cache(p, &c);
  if (st != GDN_OK) return st;
  st = check_tensors({{k, c.kin, 16, true}, {v, c.vin, 16, true}}, {{kcache, c.cache, 16, true}, {vcache, c.cache, 16, true}});
  if (st != GDN_OK || p->num_seqs == 0 || c.rows == 0) return st;
  gdn::SwaParams sp = swa_params(p, c, nullptr, k, v);
  sp.S = p->sinks; sp.slots = p->sinks + p->window; sp.kc = kcache; sp.vc = vcache;
  return hip_status(gdn::launch_swa_fill(sp, p->D, c.io == 2, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_swa_step(const gdn_swa_problem* p, const void* q, const void* k, const void* v, void* kcache, void* vcache,
                        const int32_t* lens, void* o, void* ws, size_t ws_bytes, void* stream) {
  SwaSize c;
  gdn_status st = check_cache(p, &c);
  if (st == GDN_OK) st = check_swa_grid(p, c);
  if (st != GDN_OK) return st;
  if (p->T != 1 || p->cu_seqlens_host) return GDN_ERR_SHAPE;
  st = check_tensors({{q, c.qin, 16, true}, {k, c.kin, 16, true}, {v, c.vin, 16, true}, {lens, c.lens, 4, true}},
                     {{kcache, c.cache, 16, true}, {vcache, c.cache, 16, true}, {o, c.q, 16, true}, {ws, ws_bytes, 16, false}});
  if (st != GDN_OK || p->B == 0) return st;
  if (c.step && (!ws || ws_bytes < c.step)) return GDN_ERR_WORKSPACE;
  gdn::SwaParams sp = swa_params(p, c, q, k, v);
  sp.S = p->sinks; sp.slots = p->sinks + p->window; sp.kc = kcache; sp.vc = vcache; sp.lens = lens; sp.o = o;
  sp.splits = c.splits; sp.run = c.run; sp.part = static_cast<float*>(ws);
  return hip_status(gdn::launch_swa_step(sp, p->D, c.io == 2, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
