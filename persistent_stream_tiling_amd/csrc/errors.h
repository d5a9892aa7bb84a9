// The message that gemm_last_error() returns, for every file of the C ABI.
#pragma once

namespace gsk {

// printf-style; the message belongs to the calling host thread.
void set_error(const char *fmt, ...);

}  // namespace gsk
