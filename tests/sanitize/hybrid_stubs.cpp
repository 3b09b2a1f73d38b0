// Host-only stand-ins for the device launchers of the hybrid models' operators, so that
// gdn_hybrid_abi.cpp can be built with AddressSanitizer and UndefinedBehaviorSanitizer and
// driven without a GPU.  Every launcher counts its calls and returns an error, which the ABI
// reports as GDN_ERR_HIP.
#include "gdn_hybrid.h"

extern int g_launches;

namespace gdn {
hipError_t launch_glr_fwd(const GlrParams&, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_glr_bwd(const GlrParams&, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_glr_step(const GlrParams&, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_rope_fwd(const RopeParams&, int, bool, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_rope_bwd(const RopeParams&, int, bool, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_swa_fwd(const SwaParams&, int, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_swa_bwd(const SwaParams&, int, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_swa_fill(const SwaParams&, int, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_swa_step(const SwaParams& p, int, bool, hipStream_t) {
  ++g_launches;
  // every slot belongs to one run, and no run is empty
  const bool whole = static_cast<int64_t>(p.splits) * p.run >= p.slots && static_cast<int64_t>(p.splits - 1) * p.run < p.slots;
  return whole ? hipErrorInvalidValue : hipSuccess;
}
}  // namespace gdn
