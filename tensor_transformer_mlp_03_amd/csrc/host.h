// Host-side pieces that every C entry point of the library shares: the error
// detail of the calling thread, the device check and the launch error.
#pragma once

#include <hip/hip_runtime.h>

#include <string>

#include "../../include/tpmlp.h"

namespace tpmlp {

// Detail of the calling thread's last error (tpmlp_last_error).
extern thread_local std::string g_last_error;

// Records the detail and returns the status.
tpmlp_status fail(tpmlp_status s, const std::string& what);

// TPMLP_OK if the current device is a gfx950 (cached per device).
tpmlp_status check_device();

// TPMLP_ERR_HIP with the error's text.
tpmlp_status hip_fail(hipError_t e, const char* what);

}  // namespace tpmlp
