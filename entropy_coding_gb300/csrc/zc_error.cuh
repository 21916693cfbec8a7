// zc_error.cuh — the status of a call of the runtime that failed. Launches are
// checked by the runtime's last error, which stays until it is asked for: a
// failure that is reported here is not left there for the next launch.
#pragma once

#include <cuda_runtime.h>

#include "zc.h"  // from include/ (on the -I path)

namespace zc {

inline int cuda_failed() {
    (void)cudaGetLastError();
    return ZC_ECUDA;
}

} // namespace zc
