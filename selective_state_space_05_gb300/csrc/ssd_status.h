// What the device's status words say (host code, of ssd_scan_status).
#pragma once

#include <stdio.h>

namespace ssd {

// Writes a message for the error bits of the scan's kernels and of the
// projections' into buf: of both where both are set, since a reset clears both.
// Returns whether any is.
inline bool status_message(int scan, int linear, char* buf, size_t n) {
  if (n > 0) buf[0] = 0;
  int at = 0;
  if (scan != 0)
    at = snprintf(buf, n,
                  "a tensor-core scan launch gave up a bounded wait (error bits 0x%x: 1 barrier, "
                  "2 state hand-off, 4 drain, 8 fp32 tensor-core stage); its outputs are not "
                  "valid",
                  (unsigned)scan);
  if (linear != 0 && at >= 0 && (size_t)at < n)
    snprintf(buf + at, n - at,
             "%sa projection's launch gave up a bounded wait (error bits 0x%x: 1 barrier, 2 "
             "drain); its outputs are not valid",
             at > 0 ? "; " : "", (unsigned)linear);
  return scan != 0 || linear != 0;
}

}  // namespace ssd
