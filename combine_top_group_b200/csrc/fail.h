// Errors of the calls around dispatch and combine. (Not in internal.h: the
// stored traffic of the kernels built from that file is theirs as long as it
// stays as it is.)
#pragma once

#include "ep.h"

namespace ep {

// set_last_error with a format; returns st.
ep_status_t fail(ep_status_t st, const char* fmt, ...);

}  // namespace ep
