// The calling thread's last HIP error (glu_last_hip_error), shared by the files of the C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/glu_gemv.h"

namespace glu {

// records e and returns GLU_ERR_LAUNCH
glu_status fail_launch(hipError_t e);

}  // namespace glu
