// Host-only stand-ins for the device launchers of the layer operators, so that their
// C ABI (gdn_layer_abi.cpp) can be built with AddressSanitizer and
// UndefinedBehaviorSanitizer and driven without a GPU.  Every launcher counts its calls
// and returns an error, which the ABI reports as GDN_ERR_HIP.
#include <algorithm>

#include "gdn_layer.h"

extern int g_launches;

namespace gdn {
hipError_t launch_step(const StepParams&, int, bool, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_conv_fwd(const ConvParams&, int, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_conv_bwd(const ConvParams&, int, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_conv_step(const ConvParams&, int, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_scan_fwd(const ScanParams&, int, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_scan_bwd(const ScanParams&, int, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_scan_step(const ScanParams&, int, bool, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
}  // namespace gdn
