// fa_status.cuh -- what a kernel records in its translation unit's status word, which
// fa_device_status reads.
#pragma once

#include "fa.h"

namespace fa {

// The first report stays, but that a wait ran out replaces any other: rows may then be
// unwritten, which a clamped length or a zero page does not say.
__device__ __forceinline__ void record_status(int *word, int status) {
    if (status == FA_ERR_WATCHDOG) atomicExch(word, status);
    else atomicCAS(word, 0, status);
}

}  // namespace fa
