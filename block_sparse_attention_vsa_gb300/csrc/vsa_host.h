// vsa_host.h -- host-side pieces the library's translation units share.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/vsa.h"

namespace vsa {

// The current device's ordinal (0..63); VSA_ERR_UNSUPPORTED if it is not an sm_103 device.
vsa_status host_device(int* ordinal);

// What vsa_last_launch_count() reports for this thread.
void host_set_launches(int n);

inline bool host_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool host_aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace vsa
