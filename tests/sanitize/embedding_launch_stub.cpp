// Host-only build of the embedding runtime (see launch_stub.cpp): nothing is launched.
#include "embedding_internal.h"

namespace adam_mi355x {
hipError_t launch_lookup(bool, bool, const LookupArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_group(const GroupArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_sums(bool, bool, Goal, const SumArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_direct(bool, bool, Goal, const SumArgs &, const void *, bool, hipStream_t) { return hipErrorInvalidValue; }
}  // namespace adam_mi355x
