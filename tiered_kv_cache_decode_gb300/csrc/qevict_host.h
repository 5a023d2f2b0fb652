// Error reporting and argument checks that the C entry points share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/qevict.h"

namespace qevict {

// set the calling thread's error text, return the status
qevict_status fail(qevict_status st, const char *fmt, ...);
qevict_status cuda_fail(cudaError_t e, const char *what);

struct Extent {
    const void *p;
    int64_t bytes;
    const char *what;
};
// An output must not overlap another operand: the kernels read and write in no fixed order.
inline qevict_status check_apart(const Extent &o, const Extent *others, int n) {
    const uintptr_t o0 = (uintptr_t)o.p, o1 = o0 + o.bytes;
    for (int i = 0; i < n && o.p; ++i) {
        const uintptr_t s0 = (uintptr_t)others[i].p, s1 = s0 + others[i].bytes;
        if (others[i].p && o0 < s1 && s0 < o1)
            return fail(QEVICT_ERR_INVALID_ARG, "%s overlaps %s", o.what, others[i].what);
    }
    return QEVICT_OK;
}

}  // namespace qevict
