// Host-only builds of the Muon runtime (sanitizer tests on a machine without
// a GPU): the kernel launchers are replaced by these stubs, which launch
// nothing.  The tests that use such a build only reach code that ends before
// a launch.
#include <hip/hip_runtime_api.h>

#include "muon_internal.h"

namespace adam_mi355x {
hipError_t launch_muon_momentum(int, bool, bool, const MuonStepArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_muon_norms(const double *, const uint2 *, double *, uint32_t, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_muon_sums(bool, const MuonWork &, const MuonSumArgs &, uint32_t, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_muon_prep(bool, bool, int, const MuonWork &, const MuonPrepArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_muon_product(int, int, int, int, const MuonGemmArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_muon_small(int64_t, int64_t, const MuonSmallArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_muon_decode(int, const BlockDesc *, uint32_t, const void *, const float *, void *, hipStream_t) {
    return hipErrorInvalidValue;
}
}  // namespace adam_mi355x
