// linear_dispatch.hpp - which shape of the walk runs a call (included by the files that instantiate it).
//
// bf16: 64 columns of the state a workgroup of four wavefronts, 128 where there are more (two tiles of 16 a wavefront), and
// as many stages of LDS (two or three) as leave room for a second workgroup on the CU.  fp32: 64 columns, all of LDS.
// Towards dg, where the state is twice as large, a wavefront has one tile of 16, and a workgroup of 128 columns eight wavefronts.
// With more than 128 rows those have 69 registers a lane in scratch (4 x 4096 tokens, 16 heads of 256 x 128: the backward takes 1023
// us, with four wavefronts and 64 columns, which spill none, 924); the fp32 walk of as many rows has 75.
#pragma once

#include "linear_walk.hpp"

namespace ssd {

template <typename T> constexpr int kWalkLds = (sizeof(T) == 2 ? 80 : 160) * 1024;

template <typename T, int NW, int JT, bool kOut, bool kDg>
hipError_t walk_kb(const LinearWalk<T>& p, hipStream_t stream)
{
#define SSD_WALK(KB) return launch_walk<T, KB, NW, JT, kWalkLds<T>, kOut, kDg>(p, stream)
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
            if (linear_columns(sizeof(T), p.Dv) == 128) return walk_kb<T, 8, 1, kOut, kDg>(p, stream);
        return walk_kb<T, 4, 1, kOut, kDg>(p, stream);
    } else {
        if constexpr (sizeof(T) == 2)
            if (linear_columns(sizeof(T), p.Dv) == 128) return walk_kb<T, 4, 2, kOut, kDg>(p, stream);
        return walk_kb<T, 4, 1, kOut, kDg>(p, stream);
    }
}

template <typename T, bool kOut>
hipError_t launch_linear_twin(const LinearWalk<T>& a, const LinearWalk<T>& b, hipStream_t stream)
{
#define SSD_TWIN(KB)                                                                                                   \
    do {                                                                                                               \
        if (b.Dk <= 32) return launch_twin<T, KB, 1, kWalkLds<T>, kOut>(a, b, stream);                                 \
        if (b.Dk <= 64) return launch_twin<T, KB, 2, kWalkLds<T>, kOut>(a, b, stream);                                 \
        return launch_twin<T, KB, 4, kWalkLds<T>, kOut>(a, b, stream);                                                 \
    } while (0)
    if (a.Dk <= 32) SSD_TWIN(1);
    if (a.Dk <= 64) SSD_TWIN(2);
    SSD_TWIN(4);
#undef SSD_TWIN
}

}  // namespace ssd
