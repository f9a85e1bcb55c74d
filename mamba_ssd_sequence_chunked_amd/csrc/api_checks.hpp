// api_checks.hpp - argument checks shared by the C entry points (host side, internal to the library).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "ssd.h"
#include "common.hpp"
#include "kernels.hpp"

namespace ssd {

constexpr int64_t kAlign = 256;

inline int64_t align_up(int64_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline size_t elem_size(int dtype) { return dtype == SSD_BF16 ? 2 : 4; }

inline bool valid_dtype(int dtype) { return dtype == SSD_F32 || dtype == SSD_BF16; }

inline int check_common(int64_t batch, int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups)
{
    if (batch < 0 || batch > 65535) return SSD_ERR_SHAPE;
    if (nheads < 1 || nheads > 65535) return SSD_ERR_SHAPE;
    if (headdim != 16 && headdim != 32 && headdim != 64 && headdim != 128) return SSD_ERR_SHAPE;
    if (dstate < 16 || dstate > 256 || dstate % 16 != 0) return SSD_ERR_SHAPE;
    if (ngroups < 1 || nheads % ngroups != 0) return SSD_ERR_SHAPE;
    if (nheads * headdim > (int64_t(1) << 20)) return SSD_ERR_SHAPE;   // one chunk's rows of y stay <= 2^30 bytes
    if (ngroups * dstate > (int64_t(1) << 20)) return SSD_ERR_SHAPE;   // and its rows of B and C too
    return SSD_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {
    const void* p;
    size_t bytes;
};

inline bool overlaps(Span a, Span b)
{
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

inline bool any_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins)
{
    for (const Span& o : outs) {
        for (const Span& i : ins)
            if (overlaps(o, i)) return true;
    }
    // outputs must not overlap each other either
    for (auto it = outs.begin(); it != outs.end(); ++it)
        for (auto jt = it + 1; jt != outs.end(); ++jt)
            if (overlaps(*it, *jt)) return true;
    return false;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

}  // namespace ssd
