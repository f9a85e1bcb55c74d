// linear_dispatch.hpp - which shape of the walk runs a call (included by the files that instantiate it).
//
// bf16: chunks of 64 tokens where two stages of LDS leave room for a second workgroup on the CU, else 32; 64 columns of
// the state a workgroup of four wavefronts, 128 where there are more (two tiles of 16 a wavefront).  fp32: chunks of 32,
// 64 columns.  Towards dg a wavefront has two tiles of 16, one contraction block of its share of X . V, and chunks have
// 32 tokens (twice the state in registers).
#pragma once

#include "linear_walk.hpp"

namespace ssd {

template <typename T, int KB, int NW, int JT, bool kOut, bool kDg>
constexpr int walk_chunk()
{
    return sizeof(T) == 2 && !kDg && 2 * LinearShape<T, KB, NW, JT, 64, true, false>::kStage <= 80 * 1024 ? 64 : 32;
}

template <typename T, int NW, int JT, bool kOut, bool kDg>
hipError_t walk_kb(const LinearWalk<T>& p, hipStream_t stream)
{
#define SSD_WALK(KB) return launch_walk<T, KB, NW, JT, walk_chunk<T, KB, NW, JT, kOut, kDg>(), kOut, kDg>(p, stream)
    if (p.Dk <= 32) SSD_WALK(1);
    if (p.Dk <= 64) SSD_WALK(2);
    if (p.Dk <= 128) SSD_WALK(4);
    SSD_WALK(8);
#undef SSD_WALK
}

template <typename T, bool kOut, bool kDg>
hipError_t launch_linear_walk(const LinearWalk<T>& p, hipStream_t stream)
{
    if constexpr (kDg) {
        if constexpr (sizeof(T) == 2)
            if (linear_columns(sizeof(T), true, p.Dv) == 128) return walk_kb<T, 4, 2, kOut, kDg>(p, stream);
        return walk_kb<T, 2, 2, kOut, kDg>(p, stream);
    } else {
        if constexpr (sizeof(T) == 2)
            if (linear_columns(sizeof(T), false, p.Dv) == 128) return walk_kb<T, 4, 2, kOut, kDg>(p, stream);
        return walk_kb<T, 4, 1, kOut, kDg>(p, stream);
    }
}

}  // namespace ssd
