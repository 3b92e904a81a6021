// Checks that the entry points of the operators around the mixer share
// (operators_api.hip, dense_api.hip).
#pragma once

#include "api_common.hpp"

#include <initializer_list>

namespace gdn2 {

inline hipStream_t stream() { return (hipStream_t)gdn2_get_stream(); }

inline bool dtype_ok(int t) { return t == GDN2_F32 || t == GDN2_BF16; }

// Whether an output is an input's own memory (partial overlaps are the caller's).
using Ptrs = std::initializer_list<const void *>;
inline bool same_memory(Ptrs outs, Ptrs ins)
{
    for (const void *o : outs)
        for (const void *i : ins)
            if (o && o == i) return true;
    return false;
}

// Whether two outputs are one.
inline bool twice(Ptrs outs)
{
    for (auto o = outs.begin(); o != outs.end(); ++o)
        for (auto p = outs.begin(); p != o; ++p)
            if (*o && *o == *p) return true;
    return false;
}

// Sizes whose launch would have too many threads are found where it is laid out.
inline int launch_status(hipError_t err)
{
    return err == hipSuccess ? GDN2_OK : err == hipErrorInvalidConfiguration ? GDN2_ERR_UNSUPPORTED : GDN2_ERR_HIP;
}

} // namespace gdn2
