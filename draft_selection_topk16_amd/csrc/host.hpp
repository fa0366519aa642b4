// Host-side helpers that the library's translation units share.
#pragma once

#include <hip/hip_runtime.h>

#include <string>

#include "dflash2.h"

namespace df2 {
namespace host {

#define DF2_HIDDEN __attribute__((visibility("hidden")))

// Records the message for dflash2_last_error() and returns the status.
DF2_HIDDEN df2_status fail_with(df2_status s, const std::string& msg);
DF2_HIDDEN df2_status hip_failed(hipError_t e, const char* what);
DF2_HIDDEN void clear_error();

// Compute units of the current device.
DF2_HIDDEN int compute_units();

// The current device's flag word that dflash2_device_error() reports for every
// stream (the first word of the static scratch).
DF2_HIDDEN df2_status device_flag_word(uint32_t** word);

}  // namespace host
}  // namespace df2
