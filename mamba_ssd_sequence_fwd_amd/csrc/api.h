// api.h -- what the C-ABI sources share: the thread-local error detail.
#pragma once

#include "ssd.h"

namespace ssd {

// Record a formatted detail for ssd_last_error_detail() and return `st`.
ssd_status fail(ssd_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
void clear_detail();

}  // namespace ssd
