// Host-side status reporting shared by the files that define C entry points (the text of
// ridgefill_last_error is kept per thread in ridgefill.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include "ridgefill.h"

namespace rf {

rf_status fail(rf_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
rf_status ok();
rf_status hip_fail(hipError_t e, const char* what);

}  // namespace rf
