// Host-side pieces of the C-ABI layer shared by its source files (defined in moba_api.cu).
#pragma once

#include <cuda_runtime.h>

#include "moba.h"

namespace moba {
namespace api {

void clear_error();  // of the calling thread
moba_status fail_with(moba_status st, const char* msg);
moba_status cuda_error(cudaError_t e, const char* where);
// Checks that the current device is an sm_100 part and gives its device error word.
moba_status device_error_word(int** err);

}  // namespace api
}  // namespace moba
