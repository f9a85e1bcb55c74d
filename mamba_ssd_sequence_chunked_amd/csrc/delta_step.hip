// delta_step.hip - the gated delta rule's recurrent mode: one token per call, state updated in place.
//
//   S' = exp(g) S;  e[p] = v[p] - sum_n S'[p, n] k[n];  u = beta e;  S[p, n] = S'[p, n] + u[p] k[n]
//   y[p] = sum_n S[p, n] q[n] = sum_n S'[p, n] q[n] + u[p] (k . q)
//
// Written with the second form of y, both sums over a state row need the decayed state only, so one
// pass over the row gives them together and the updated row leaves right after.  The fp32 state is
// read and written once and there are 7 flops per state element: the kernel is bound by HBM bandwidth.
//
// Workgroup = one (batch, head): its P x N state block is contiguous.  A thread owns 4 consecutive
// columns (one 16-byte vector) of every (256 / W)-th row, W lanes to a row (a power of two >= N / 4;
// surplus lanes contribute 0).  All rows are loaded before any arithmetic, non-temporal, as in ssd_step.
// Measured: 256 rows of 80 heads of 64 x 128 (bf16) 234 us, 5.8 TB/s of state; 13 rows of 20 heads of 128 x 256 (fp32)
// 20 us; one row of 24 heads 6.3 us.
#include "common.hpp"
#include "kernels.hpp"

namespace ssd {

namespace {

template <typename T, int W, int P>
__global__ __launch_bounds__(256) void delta_step_kernel(
    float* __restrict__ state, const T* __restrict__ v, const float* __restrict__ gv, const float* __restrict__ bv,
    const T* __restrict__ Km, const T* __restrict__ Qm, T* __restrict__ y, int nheads, int N, int ngroups)
{
    constexpr int kRowsPerPass = 256 / W;
    constexpr int kPass = (P + kRowsPerPass - 1) / kRowsPerPass;
    const int bh = blockIdx.x;
    const int h = bh % nheads;
    const int b = bh / nheads;
    const int grp = h / (nheads / ngroups);
    const int tid = threadIdx.x;
    const int col = 4 * (tid % W);
    const int rsub = tid / W;
    const bool colok = col < N;

    const float a = __expf(gv[bh]);
    const float beta = bv[bh];
    float kv[4] = {0.f, 0.f, 0.f, 0.f}, qv[4] = {0.f, 0.f, 0.f, 0.f};
    if (colok) {
        const T* kp = Km + ((int64_t)b * ngroups + grp) * N + col;
        const T* qp = Qm + ((int64_t)b * ngroups + grp) * N + col;
#pragma unroll
        for (int e = 0; e < 4; ++e) { kv[e] = to_f32(kp[e]); qv[e] = to_f32(qp[e]); }
    }
    float* S = state + (int64_t)bh * P * N;
    const T* vr = v + (int64_t)bh * P;
    T* yr = y + (int64_t)bh * P;
    float4 s[kPass];
    float vv[kPass];
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
        const int p = i * kRowsPerPass + rsub;
        const bool live = p < P;
        vv[i] = live ? to_f32(vr[p]) : 0.f;
        f32x4 t4 = f32x4{0.f, 0.f, 0.f, 0.f};
        if (live && colok) t4 = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + (int64_t)p * N + col));
        s[i] = make_float4(t4[0], t4[1], t4[2], t4[3]);
    }
    const float kq = group_sum<W>(kv[0] * qv[0] + kv[1] * qv[1] + kv[2] * qv[2] + kv[3] * qv[3]);
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
        const int p = i * kRowsPerPass + rsub;
        const bool live = p < P;
        float4 t = s[i];
        t.x *= a; t.y *= a; t.z *= a; t.w *= a;
        const float sk = group_sum<W>(t.x * kv[0] + t.y * kv[1] + t.z * kv[2] + t.w * kv[3]);
        const float sq = group_sum<W>(t.x * qv[0] + t.y * qv[1] + t.z * qv[2] + t.w * qv[3]);
        const float u = beta * (vv[i] - sk);
        if (live && colok)
            __builtin_nontemporal_store(f32x4{fmaf(u, kv[0], t.x), fmaf(u, kv[1], t.y), fmaf(u, kv[2], t.z),
                                              fmaf(u, kv[3], t.w)},
                                        reinterpret_cast<f32x4*>(S + (int64_t)p * N + col));
        if ((tid % W) == 0 && live) yr[p] = from_f32<T>(fmaf(u, kq, sq));
    }
}

template <typename T, int W, int P>
hipError_t launch(float* state, const T* v, const float* g, const float* beta, const T* k, const T* q, T* y,
                  const DeltaDims& d, hipStream_t stream)
{
    const int64_t nblocks = d.seqs * d.nheads;
    if (nblocks == 0) return hipSuccess;
    hipLaunchKernelGGL((delta_step_kernel<T, W, P>), dim3((unsigned)nblocks), dim3(256), 0, stream, state, v, g, beta,
                       k, q, y, (int)d.nheads, (int)d.dstate, (int)d.ngroups);
    return hipGetLastError();
}

template <typename T, int W>
hipError_t launch_w(float* state, const T* v, const float* g, const float* beta, const T* k, const T* q, T* y,
                    const DeltaDims& d, hipStream_t stream)
{
    switch (d.headdim) {
    case 16: return launch<T, W, 16>(state, v, g, beta, k, q, y, d, stream);
    case 32: return launch<T, W, 32>(state, v, g, beta, k, q, y, d, stream);
    case 64: return launch<T, W, 64>(state, v, g, beta, k, q, y, d, stream);
    case 128: return launch<T, W, 128>(state, v, g, beta, k, q, y, d, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

template <typename T>
hipError_t launch_delta_step(float* state, const T* v, const float* g, const float* beta, const T* k, const T* q,
                             T* y, const DeltaDims& d, hipStream_t stream)
{
    const int64_t w = d.dstate / 4;
    if (w <= 4) return launch_w<T, 4>(state, v, g, beta, k, q, y, d, stream);
    if (w <= 8) return launch_w<T, 8>(state, v, g, beta, k, q, y, d, stream);
    if (w <= 16) return launch_w<T, 16>(state, v, g, beta, k, q, y, d, stream);
    if (w <= 32) return launch_w<T, 32>(state, v, g, beta, k, q, y, d, stream);
    return launch_w<T, 64>(state, v, g, beta, k, q, y, d, stream);
}

template hipError_t launch_delta_step<float>(float*, const float*, const float*, const float*, const float*,
                                             const float*, float*, const DeltaDims&, hipStream_t);
template hipError_t launch_delta_step<bf16>(float*, const bf16*, const float*, const float*, const bf16*, const bf16*,
                                            bf16*, const DeltaDims&, hipStream_t);

}  // namespace ssd
