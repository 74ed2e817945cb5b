// Calls between libpa.so and the Python binding's module that are not part of the C interface.
#pragma once

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

// The id of the capture that `stream` takes part in, which no other capture of the process
// has; 0 outside one.
unsigned long long pa_stream_capture_id(pa_stream_t stream);

#ifdef __cplusplus
}
#endif
