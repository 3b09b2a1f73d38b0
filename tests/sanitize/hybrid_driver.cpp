// Drives the C ABI of gdn_glr_*, gdn_rope_* and gdn_swa_* under the sanitizers: sizes over a
// grid of problems up to the documented limits and past them, and every entry point with NULL
// and with valid-looking arguments (addresses are never dereferenced: the launchers are stubs).
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "gdn.h"

extern int g_launches;

static int g_checks = 0;
#define CHECK(x)                                                   \
  do {                                                             \
    ++g_checks;                                                    \
    if (!(x)) {                                                    \
      std::printf("failed: %s (line %d)\n", #x, __LINE__);         \
      std::exit(1);                                                \
    }                                                              \
  } while (0)

// far enough apart for the largest tensor
static void* at(int i) { return reinterpret_cast<void*>((static_cast<uintptr_t>(i) + 1) << 54); }
static float* fat(int i) { return static_cast<float*>(at(i)); }
static const int32_t* iat(int i) { return static_cast<const int32_t*>(at(i)); }
static const size_t kAll = static_cast<size_t>(1) << 53;

static bool known(gdn_status st) {
  return st == GDN_OK || st == GDN_ERR_HIP || st == GDN_ERR_SHAPE || st == GDN_ERR_UNSUPPORTED || st == GDN_ERR_DTYPE ||
         st == GDN_ERR_ALIGN || st == GDN_ERR_SEQLENS;
}

static void glr(const gdn_glr_problem& p) {
  size_t f = 0, s = 0, b = 0;
  const gdn_status st = gdn_glr_workspace_size(&p, GDN_GLR_FWD, &f);
  CHECK(known(st) && gdn_glr_workspace_size(&p, GDN_GLR_SAVED, &s) == st && gdn_glr_workspace_size(&p, GDN_GLR_BWD, &b) == st);
  const gdn_status run = gdn_glr_fwd(&p, at(0), at(1), at(2), fat(3), at(4), fat(5), at(6), fat(7), at(8), f, nullptr);
  CHECK(st == GDN_OK ? run == (p.num_seqs ? GDN_ERR_HIP : GDN_OK) : run == st);
  CHECK(known(gdn_glr_fwd_save(&p, at(0), at(1), at(2), fat(3), nullptr, nullptr, at(6), nullptr, at(9), s, at(8), f, nullptr)));
  CHECK(known(gdn_glr_bwd_saved(&p, at(0), at(1), at(2), fat(3), at(4), at(10), fat(11), at(9), s, at(12), at(13), at(14), fat(15), at(16),
                                fat(17), at(8), b, nullptr)));
  CHECK(known(gdn_glr_step(&p, at(0), at(1), at(2), fat(3), nullptr, fat(5), at(6), nullptr)));
}

static void rope(const gdn_rope_problem& p) {
  size_t n = 0;
  const gdn_status st = gdn_rope_workspace_size(&p, &n);
  CHECK(known(st));
  const bool rms = p.norm == GDN_ROPE_RMS, none = p.B <= 0 || p.T <= 0;
  const gdn_status run = gdn_rope_fwd(&p, at(0), at(1), fat(2), iat(3), rms ? fat(4) : nullptr, nullptr, at(5), at(6), nullptr);
  CHECK(st == GDN_OK ? run == (none ? GDN_OK : GDN_ERR_HIP) : run == st);
  CHECK(known(gdn_rope_bwd(&p, at(0), at(1), fat(2), nullptr, nullptr, rms ? fat(4) : nullptr, at(5), at(6), at(7), at(8),
                           rms ? fat(9) : nullptr, rms ? fat(10) : nullptr, at(11), n, nullptr)));
}

static void swa(const gdn_swa_problem& p) {
  size_t b = 0, s = 0;
  const gdn_status st = gdn_swa_workspace_size(&p, GDN_SWA_BWD, &b);
  const gdn_status sc = gdn_swa_workspace_size(&p, GDN_SWA_STEP, &s);
  CHECK(known(st) && known(sc) && (st == GDN_OK || sc == st));
  const bool none = p.B <= 0 || p.T <= 0;
  const gdn_status run = gdn_swa_fwd(&p, at(0), at(1), at(2), at(3), fat(4), nullptr);
  CHECK(st == GDN_OK ? run == (none ? GDN_OK : GDN_ERR_HIP) : run == st);
  CHECK(known(gdn_swa_bwd(&p, at(0), at(1), at(2), at(3), fat(4), at(5), at(6), at(7), at(8), at(9), b, nullptr)));
  CHECK(known(gdn_swa_fill(&p, at(1), at(2), at(10), at(11), nullptr)));
  const gdn_status step = gdn_swa_step(&p, at(0), at(1), at(2), at(10), at(11), iat(12), at(3), at(9), s, nullptr);
  if (sc == GDN_OK) CHECK(p.T != 1 || p.cu_seqlens_host ? step == GDN_ERR_SHAPE : step == (p.B ? GDN_ERR_HIP : GDN_OK));
}

int main() {
  const int32_t sizes[] = {-1, 0, 1, 7, 64, 129, 4096, 65535, 65536, 1 << 20, INT32_MAX};
  for (int32_t B : sizes)
    for (int32_t T : sizes)
      for (int dt : {0, 1, 2}) {
        for (int32_t C : {0, 8, 12, 64, 2056, 1 << 20, (1 << 20) + 8, INT32_MAX})
          glr(gdn_glr_problem{B, T, C, B, nullptr, nullptr, dt, 8.f});
        for (int32_t H : {0, 1, 16, 4096, INT32_MAX})
          for (int32_t D : {0, 64, 128, 256, INT32_MAX}) {
            for (int norm : {0, 1, 2, 3})
              rope(gdn_rope_problem{B, T, H, 1, D, D == INT32_MAX ? 0 : D, norm, 1, dt, 1e-6f, 0, 0});
            rope(gdn_rope_problem{B, T, H, H, D, 16, 1, 0, dt, 1e-6f, INT64_MAX, 1 << 21});
            for (int32_t W : {0, 1, 4096, 1 << 30, INT32_MAX})
              for (int32_t S : {0, 1, 1024, INT32_MAX}) {
                swa(gdn_swa_problem{B, T, H, 1, D, W, S, B, nullptr, nullptr, dt, 1.f, 0, 0, 0});
                swa(gdn_swa_problem{B, T, H, H, D, W, S, B, nullptr, nullptr, dt, 1.f, INT64_MAX, 1 << 21, INT64_MIN});
              }
          }
      }
  // packed: ragged offsets, then every way they can be wrong
  std::vector<int32_t> cu = {0, 0, 3, 3, 900};
  gdn_glr_problem g{1, 900, 64, 4, cu.data(), iat(30), GDN_BF16, 8.f};
  gdn_swa_problem w{1, 900, 4, 2, 64, 100, 5, 4, cu.data(), iat(30), GDN_BF16, 1.f, 0, 0, 0};
  glr(g);
  swa(w);
  CHECK(gdn_glr_fwd(&g, at(0), at(1), at(2), fat(3), nullptr, nullptr, at(6), nullptr, at(8), kAll, nullptr) == GDN_ERR_HIP);
  for (int i : {0, 2, 4}) {
    const int32_t keep = cu[i];
    cu[i] = 1000;
    size_t n = 0;
    CHECK(gdn_glr_workspace_size(&g, GDN_GLR_BWD, &n) == GDN_ERR_SEQLENS && gdn_swa_workspace_size(&w, GDN_SWA_BWD, &n) == GDN_ERR_SEQLENS);
    cu[i] = keep;
  }
  size_t n = 0;
  CHECK(gdn_glr_workspace_size(nullptr, GDN_GLR_FWD, &n) == GDN_ERR_NULL && gdn_glr_workspace_size(&g, GDN_GLR_FWD, nullptr) == GDN_ERR_NULL);
  CHECK(gdn_rope_workspace_size(nullptr, &n) == GDN_ERR_NULL && gdn_swa_workspace_size(nullptr, GDN_SWA_BWD, &n) == GDN_ERR_NULL);
  CHECK(gdn_glr_workspace_size(&g, 3, &n) == GDN_ERR_UNSUPPORTED && gdn_swa_workspace_size(&w, -1, &n) == GDN_ERR_UNSUPPORTED);
  std::printf("ok: %d checks, %d launches\n", g_checks, g_launches);
  return 0;
}
