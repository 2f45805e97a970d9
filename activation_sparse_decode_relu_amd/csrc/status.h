// The status and message every C entry point returns with (internal to the library).
#pragma once

#include "pi_ffn.h"

namespace pik {

// Keep the printf-style message as this thread's last error; returns st.
pi_status fail(pi_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// Clear this thread's last error; returns PI_OK.
pi_status ok();

}  // namespace pik
