// Host-side internals of the calls around dispatch and combine. (Not in
// internal.h: the stored traffic of the kernels built from that file is theirs
// as long as it stays as it is.)
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ep.h"

namespace ep {

// set_last_error with a format; returns st.
ep_status_t fail(ep_status_t st, const char* fmt, ...);

// The linear layers' waits and drains on a phase that never completes; sets
// *gave_up = 1 and EP_DEVERR_TIMEOUT in *err when each of them has ended unmet.
cudaError_t launch_linear_timeout_selftest(uint32_t* err, uint32_t* gave_up, unsigned long long limit_ns,
                                           cudaStream_t stream);

}  // namespace ep
