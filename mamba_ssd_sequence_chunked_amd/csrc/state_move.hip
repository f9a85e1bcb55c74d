// state_move.hip - states of a pool copied, forked, reordered and freed by one map of slots, in place.
//
//   states[l, i] = source[l, src[i]]    where 0 <= src[i] < nsource (in place: the states as they were, and src[i] != i)
//   states[l, i] = 0                    where src[i] == -1
//   states[l, i] stays                  else
//
// Only copies: bound by HBM bandwidth (180 of 256 slots of 2.6 MB taken from 110 others, 4 cleared: 156 to 161 us, 4.9 TB/s;
// the smallest moves 10 us, of which half are the scan of the map and one wait for memory).  In place any map is allowed (a slot may be read by others and overwritten itself), with
// no copy of the pool and no order to be found: slots do not mix columns, so a workgroup takes a strip of columns of ALL
// moves, reads them into registers, waits until all its wavefronts have, and writes them.  16 wavefronts with 8 vectors
// of 16 bytes a lane hold 128 moves of 1 KB strips; more moves take strips of 256 or 64 bytes (512, 2048 moves), and
// fewer moves several strips at once.  Between two pools nothing is overwritten that is read, and more moves go in turns.
#include "common.hpp"
#include "kernels.hpp"

namespace ssd {

namespace {

constexpr int kWaves = 16, kHeld = 8, kScan = 2048;

__global__ __launch_bounds__(kWaves * 64) void state_move_kernel(float* states, const float* source,
                                                                 const int32_t* __restrict__ src, int64_t nlayers,
                                                                 int nslots, int nsource, int64_t quads)
{
    __shared__ int to[kScan], from[kScan], count[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const bool in_place = source == states;
    const int64_t strips = (quads + 63) / 64, all = strips * nlayers;
    const int64_t begin = all * blockIdx.x / gridDim.x, end = all * (blockIdx.x + 1) / gridDim.x;

    for (int slot0 = 0; slot0 < nslots; slot0 += kScan) {
        // the moves among kScan slots, in their order: two slots a thread
        int m[2], n = 0;
        bool moves[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = slot0 + 2 * tid + k;
            m[k] = i < nslots ? src[i] : nsource;
            moves[k] = m[k] >= -1 && m[k] < nsource && !(in_place && m[k] == i);
            n += moves[k];
        }
        const int before = (int)wave_inclusive_sum((float)n) - n;      // (small whole numbers: exact)
        if (lane == 63) count[wave] = before + n;
        __syncthreads();
        int at = before, total = 0;
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) at += count[w];
            total += count[w];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (moves[k]) { to[at] = slot0 + 2 * tid + k; from[at] = m[k]; ++at; }
        __syncthreads();
        if (total > 0) {
            // lanes to a move, moves to a vector instruction, strips at once
            const int lp = total <= kWaves * kHeld ? 64 : total <= 4 * kWaves * kHeld ? 16 : 4;
            const int rp = 64 / lp, groups = (total + rp - 1) / rp, sp = max(kWaves * kHeld / groups, 1);
            for (int64_t s0 = begin * rp; s0 < end * rp; s0 += sp) {
                const int cnt = (int)min((int64_t)sp, end * rp - s0), items = groups * cnt;
                f32x4 held[kHeld];
                int64_t where[kHeld];                              // the destination's quad, or -1
#pragma unroll
                for (int i = 0; i < kHeld; ++i) {
                    const int e = wave + kWaves * i;
                    where[i] = -1;
                    held[i] = f32x4{0.f, 0.f, 0.f, 0.f};
                    const int row = (e / cnt) * rp + lane / lp;
                    const int64_t strip = s0 + e % cnt, layer = strip / (strips * rp);
                    const int64_t q = (strip - layer * strips * rp) * lp + lane % lp;
                    if (e < items && row < total && q < quads) {
                        where[i] = (layer * nslots + to[row]) * quads + q;
                        if (from[row] >= 0)
                            held[i] = reinterpret_cast<const f32x4*>(source)[(layer * nsource + from[row]) * quads + q];
                    }
                }
                wait_vmem();                                       // read, not only asked for
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kHeld; ++i)
                    if (where[i] >= 0) reinterpret_cast<f32x4*>(states)[where[i]] = held[i];
            }
        }
        __syncthreads();
    }
}

}  // namespace

hipError_t launch_state_move(float* states, const float* source, const int32_t* src, int64_t nlayers, int64_t nslots,
                             int64_t nsource, int64_t slot_floats, hipStream_t stream)
{
    const int64_t strips = (slot_floats / 4 + 63) / 64 * nlayers;
    if (strips == 0 || nslots == 0) return hipSuccess;
    // One workgroup to a CU where moves are few, with which starting it is most of its time (4 of 16 slots forked in 4 layers:
    // 256 workgroups 9.9 us, the host's share; 512 14.8; 1024 24.4), two where a pool is large (180 of 256 states of
    // 2.6 MB: 168, 164, 174).
    const int64_t most = nslots <= 64 ? 256 : 512, blocks = strips < most ? strips : most;
    hipLaunchKernelGGL(state_move_kernel, dim3((unsigned)blocks), dim3(kWaves * 64), 0, stream, states,
                       source ? source : states, src, nlayers, (int)nslots, (int)nsource, slot_floats / 4);
    return hipGetLastError();
}

}  // namespace ssd
