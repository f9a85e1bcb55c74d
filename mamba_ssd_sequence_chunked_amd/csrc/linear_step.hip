// linear_step.hip - linear attention with a decay for each head, one token per call, states updated in place.
//
//   S[p, n] = a S[p, n] + v[p] k[n];   y[p] = sum_n S[p, n] q[n],   a = exp(g)
//
// The fp32 state is read and written once, 5 flops an element: bound by HBM bandwidth (240 of 256 rows, 80 heads of 64 x 128:
// 227 to 233 us, 5.5 TB/s; 13 rows, 20 heads of 128 x 256 13.7 us, 5.0 TB/s).  One row of 24 heads is the launch, 6 us.  A thread owns 4
// consecutive columns of every (256 / W)-th row, W lanes to a row (a power of two >= N / 4; surplus lanes contribute 0),
// and kPass rows; a workgroup has kPass * 256 / W rows of one (batch row, head).  All its rows are on the way before any
// arithmetic, non-temporal, as in ssd_step.  Large heads take several workgroups: with one each a CU's reads and
// writes would not overlap.
//
// With slots a row's state is slots[row] of a pool.  A slot out of range is no state (padding): its row's y is zero.  A slot
// that an earlier row has is taken as out of range: two rows never touch one state, whatever the table holds.
#include "common.hpp"
#include "kernels.hpp"

namespace ssd {

namespace {

template <typename T, int W, int kPass>
__global__ __launch_bounds__(256) void linear_step_kernel(
    float* __restrict__ state, const int32_t* __restrict__ slots, int64_t nslots, const T* __restrict__ v,
    const float* __restrict__ gv, const T* __restrict__ Km, const T* __restrict__ Qm, T* __restrict__ y, int nheads,
    int P, int N, int ngroups, int parts)
{
    constexpr int kRows = 256 / W;
    const int bh = blockIdx.x / parts, p0 = (blockIdx.x % parts) * (kRows * kPass);
    const int h = bh % nheads, b = bh / nheads;
    const int tid = threadIdx.x, col = 4 * (tid % W), rsub = tid / W;
    const bool colok = col < N;
    const int64_t grp = (int64_t)b * ngroups + h / (nheads / ngroups);

    int64_t slot = b;
    bool ok = true;
    if (slots) {
        slot = slots[b];
        ok = slot >= 0 && slot < nslots;
    }
    float* S = state + (slot * nheads + h) * (int64_t)P * N;
    f32x4 s[kPass];
    float vv[kPass];
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
        const int p = p0 + i * kRows + rsub;
        const bool live = p < P;
        vv[i] = live ? to_f32(v[grp * P + p]) : 0.f;
        s[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (ok && live && colok) s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + (int64_t)p * N + col));
    }
    const float a = expf(linear_rate(gv[h]));
    float kv[4] = {0.f, 0.f, 0.f, 0.f}, qv[4] = {0.f, 0.f, 0.f, 0.f};
    if (colok) {
        const float4 k4 = load4f(Km + grp * N + col), q4 = load4f(Qm + (int64_t)bh * N + col);
        kv[0] = k4.x; kv[1] = k4.y; kv[2] = k4.z; kv[3] = k4.w;
        qv[0] = q4.x; qv[1] = q4.y; qv[2] = q4.z; qv[3] = q4.w;
    }
    if (slots) {
        bool before = false;
        for (int j = tid; j < b; j += 256) before |= slots[j] == slot;
        ok = !__syncthreads_or(before) && ok;
    }
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
        const int p = p0 + i * kRows + rsub;
        const bool live = p < P;
#pragma unroll
        for (int m = 0; m < 4; ++m) s[i][m] = fmaf(a, s[i][m], vv[i] * kv[m]);
        const float sq = group_sum<W>(s[i][0] * qv[0] + s[i][1] * qv[1] + s[i][2] * qv[2] + s[i][3] * qv[3]);
        if (ok && live && colok) __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(S + (int64_t)p * N + col));
        if ((tid % W) == 0 && live) y[(int64_t)bh * P + p] = from_f32<T>(ok ? sq : 0.f);
    }
}

template <typename T, int W>
hipError_t launch_w(float* state, const int32_t* slots, int64_t nslots, const T* v, const float* g, const T* k, const T* q,
                    T* y, const DeltaDims& d, hipStream_t stream)
{
    constexpr int kRows = 256 / W;
    const int P = (int)d.headdim;
#define SSD_STEP(PASS)                                                                                                 \
    do {                                                                                                               \
        const int parts = (P + kRows * PASS - 1) / (kRows * PASS);                                                     \
        hipLaunchKernelGGL((linear_step_kernel<T, W, PASS>), dim3((unsigned)(d.seqs * d.nheads * parts)), dim3(256), 0, \
                           stream, state, slots, nslots, v, g, k, q, y, (int)d.nheads, P, (int)d.dstate,                \
                           (int)d.ngroups, parts);                                                                     \
        return hipGetLastError();                                                                                      \
    } while (0)
    if (P <= kRows) SSD_STEP(1);
    if (P <= 2 * kRows) SSD_STEP(2);
    if (P <= 4 * kRows) SSD_STEP(4);
    SSD_STEP(8);
#undef SSD_STEP
}

}  // namespace

template <typename T>
hipError_t launch_linear_step(float* state, const int32_t* slots, int64_t nslots, const T* v, const float* g, const T* k,
                              const T* q, T* y, const DeltaDims& d, hipStream_t stream)
{
    const int64_t w = d.dstate / 4;
    if (w <= 4) return launch_w<T, 4>(state, slots, nslots, v, g, k, q, y, d, stream);
    if (w <= 8) return launch_w<T, 8>(state, slots, nslots, v, g, k, q, y, d, stream);
    if (w <= 16) return launch_w<T, 16>(state, slots, nslots, v, g, k, q, y, d, stream);
    if (w <= 32) return launch_w<T, 32>(state, slots, nslots, v, g, k, q, y, d, stream);
    return launch_w<T, 64>(state, slots, nslots, v, g, k, q, y, d, stream);
}

template hipError_t launch_linear_step<float>(float*, const int32_t*, int64_t, const float*, const float*, const float*,
                                              const float*, float*, const DeltaDims&, hipStream_t);
template hipError_t launch_linear_step<bf16>(float*, const int32_t*, int64_t, const bf16*, const float*, const bf16*,
                                             const bf16*, bf16*, const DeltaDims&, hipStream_t);

}  // namespace ssd
