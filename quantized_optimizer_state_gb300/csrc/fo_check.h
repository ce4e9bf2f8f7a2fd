// fo_check.h -- checks of arguments that the C-ABI layers of the losses and of the
// operators on activations share. Not installed; not part of the ABI.
#pragma once

#include <cstdint>

#include "fo.h"

namespace fo {
namespace check {

inline int64_t element_size(int32_t dtype) { return dtype == FO_LOGITS_F32 ? 4 : 2; }
inline bool dtype_ok(int32_t dtype) { return dtype == FO_LOGITS_BF16 || dtype == FO_LOGITS_F32 || dtype == FO_LOGITS_F16; }
inline bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// One array of a call: bytes [lo, hi), empty where the pointer is null.
struct Range {
    uintptr_t lo = 0, hi = 0;
    bool written = false;
    Range() = default;
    Range(const void *p, int64_t bytes, bool w) : lo(reinterpret_cast<uintptr_t>(p)), hi(lo), written(w)
    {
        if (p)
            hi = lo + (uintptr_t)bytes;
    }
};

// A written array may share no byte with any other array of the call.
inline bool aliases(const Range *r, int n)
{
    for (int a = 0; a < n; ++a)
        for (int b = a + 1; b < n; ++b)
            if ((r[a].written || r[b].written) && r[a].lo < r[b].hi && r[b].lo < r[a].hi)
                return true;
    return false;
}

}  // namespace check
}  // namespace fo
