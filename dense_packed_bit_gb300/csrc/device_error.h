// device_error.h -- what a device error word says that holds both kinds of events, as the 4-bit products' do.
//
// A kernel adds its events to the word with atomicOr: codes of waits that ran out lie below kRangeBit, a bit of its own, so
// neither kind hides the other.
#pragma once

#include "mm.h"

namespace mm {

constexpr unsigned int kRangeBit = 16;

// A wait that ran out comes first: what the call wrote is then wrong whatever its arguments were.
inline mm_status device_error_status(unsigned int word) {
    if (word & ~kRangeBit) return MM_ERR_TIMEOUT;
    return word ? MM_ERR_INVALID_ARG : MM_OK;
}

}  // namespace mm
