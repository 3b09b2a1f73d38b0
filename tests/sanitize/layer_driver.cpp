// Drives the layer operators' C ABI under the sanitizers: workspace sizes over a grid of
// problems up to the documented limits, and every entry point with NULL and with
// valid-looking arguments (addresses are never dereferenced: the launchers are stubs).
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

static void* at(int i) { return reinterpret_cast<void*>(static_cast<uintptr_t>(0x100000000000ull) + (static_cast<uintptr_t>(i) << 40)); }
static float* fat(int i) { return static_cast<float*>(at(i)); }

int main() {
  const int32_t sizes[] = {-1, 0, 1, 2, 7, 8, 64, 4096, 65535, 65536, 1 << 20, INT32_MAX};
  const int32_t chans[] = {0, 8, 12, 64, 2056, 1 << 20, (1 << 20) + 8, INT32_MAX};
  for (int32_t B : sizes)
    for (int32_t T : sizes)
      for (int32_t C : chans)
        for (int32_t w : {0, 2, 4, 5})
          for (int dt : {0, 1, 2}) {
            size_t n = 0;
            gdn_conv_problem p{B, T, C, w, B, nullptr, nullptr, dt, GDN_ACT_SILU};
            if (gdn_conv_workspace_size(&p, &n) == GDN_OK) {
              CHECK(n <= (static_cast<size_t>(B) * T / 512 + 1) * C * 5 * 4);
              const int before = g_launches;
              const gdn_status st = gdn_conv_fwd(&p, at(1), fat(2), nullptr, nullptr, at(3), nullptr, nullptr);
              CHECK(st == (B == 0 ? GDN_OK : GDN_ERR_HIP) && g_launches == before + (B != 0));
            }
            for (int32_t N : {0, 8, 16, 64, 65})
              for (int32_t G : {0, 1, 4}) {
                gdn_scan_problem s{B, T, C, N, G, B, nullptr, nullptr, dt, 1};
                size_t a = 0, b = 0, c = 0;
                const gdn_status st = gdn_scan_workspace_size(&s, GDN_SCAN_FWD, &a);
                CHECK(gdn_scan_workspace_size(&s, GDN_SCAN_SAVED, &b) == st);
                CHECK(gdn_scan_workspace_size(&s, GDN_SCAN_BWD, &c) == st);
                if (st == GDN_OK && B > 0) CHECK(b >= static_cast<size_t>(B) * T / 16 * C * N * 4);
              }
          }
  // packed: ragged offsets, then every way they can be wrong
  std::vector<int32_t> cu = {0, 0, 3, 3, 40};
  gdn_scan_problem s{1, 40, 64, 16, 2, 4, cu.data(), static_cast<const int32_t*>(at(30)), GDN_BF16, 1};
  size_t nf = 0, ns = 0, nb = 0;
  CHECK(gdn_scan_workspace_size(&s, GDN_SCAN_FWD, &nf) == GDN_OK);
  CHECK(gdn_scan_workspace_size(&s, GDN_SCAN_SAVED, &ns) == GDN_OK);
  CHECK(gdn_scan_workspace_size(&s, GDN_SCAN_BWD, &nb) == GDN_OK);
  CHECK(gdn_scan_fwd(&s, at(1), at(2), fat(3), at(4), at(5), nullptr, nullptr, nullptr, nullptr, at(6), nullptr, at(7), nf, nullptr) == GDN_ERR_HIP);
  CHECK(gdn_scan_fwd_save(&s, at(1), at(2), fat(3), at(4), at(5), fat(8), at(9), fat(10), fat(11), at(6), fat(12), at(13), ns, at(7), nf, nullptr) == GDN_ERR_HIP);
  CHECK(gdn_scan_bwd_saved(&s, at(1), at(2), fat(3), at(4), at(5), fat(8), at(9), fat(10), at(14), fat(15), at(13), ns, at(16), at(17), fat(18),
                           at(19), at(20), fat(21), at(22), fat(23), fat(24), at(7), nb, nullptr) == GDN_ERR_HIP);
  CHECK(gdn_scan_step(&s, at(1), at(2), fat(3), at(4), at(5), nullptr, nullptr, nullptr, fat(6), at(7), nullptr) == GDN_ERR_SHAPE);
  cu[2] = 50;
  CHECK(gdn_scan_workspace_size(&s, GDN_SCAN_FWD, &nf) == GDN_ERR_SEQLENS);
  CHECK(gdn_scan_workspace_size(nullptr, GDN_SCAN_FWD, &nf) == GDN_ERR_NULL);
  CHECK(gdn_scan_workspace_size(&s, GDN_SCAN_FWD, nullptr) == GDN_ERR_NULL);
  gdn_conv_problem c{3, 1, 64, 4, 3, nullptr, nullptr, GDN_BF16, GDN_ACT_NONE};
  CHECK(gdn_conv_step(&c, at(1), fat(2), nullptr, at(3), at(4), nullptr) == GDN_ERR_HIP);
  CHECK(gdn_conv_step(nullptr, at(1), fat(2), nullptr, at(3), at(4), nullptr) == GDN_ERR_NULL);
  size_t nc = 0;
  CHECK(gdn_conv_workspace_size(&c, &nc) == GDN_OK);
  CHECK(gdn_conv_bwd(&c, at(1), fat(2), fat(3), at(4), at(5), at(6), at(7), fat(8), fat(9), at(10), at(11), nc, nullptr) == GDN_ERR_HIP);
  gdn_problem p{2, 1, 3, 64, 48, 2, nullptr, nullptr, GDN_BF16, 1.f, 64, 1, 0};
  CHECK(gdn_step(&p, at(1), at(2), at(3), fat(4), fat(5), fat(6), at(7), nullptr) == GDN_ERR_HIP);
  CHECK(gdn_kda_step(&p, at(1), at(2), at(3), fat(4), fat(5), fat(6), at(7), nullptr) == GDN_ERR_HIP);
  CHECK(gdn_step(nullptr, at(1), at(2), at(3), fat(4), fat(5), fat(6), at(7), nullptr) == GDN_ERR_NULL);
  p.B = p.num_seqs = 0;
  CHECK(gdn_step(&p, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr) == GDN_OK);
  std::printf("ok: %d checks, %d launches\n", g_checks, g_launches);
  return 0;
}
