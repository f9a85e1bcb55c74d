// delta_fwd.hip - the gated delta rule over whole sequences, token by token.
//
//   S' = exp(g_t) S;  e = v_t - S' k_t;  S = S' + beta_t e k_t^T;  y_t = S q_t
//
// The recurrence as it stands: a workgroup holds one (sequence, head)'s P x N state in registers (a thread
// owns 4 columns of every (256 / W)-th row) and walks the tokens.
#include "common.hpp"
#include "kernels.hpp"

namespace ssd {

namespace {

template <typename T, int W, int P>
__global__ __launch_bounds__(256) void delta_fwd_kernel(
    const T* __restrict__ v, const float* __restrict__ gv, const float* __restrict__ bv, const T* __restrict__ Km,
    const T* __restrict__ Qm, const float* __restrict__ init, T* __restrict__ y, float* __restrict__ fin,
    const int32_t* __restrict__ cu, int64_t seqlen, int64_t tokens, int nheads, int N, int ngroups)
{
    constexpr int kRowsPerPass = 256 / W;
    constexpr int kPass = (P + kRowsPerPass - 1) / kRowsPerPass;
    const int64_t sh = blockIdx.x;
    const int h = (int)(sh % nheads);
    const int64_t s = sh / nheads;
    const int grp = h / (nheads / ngroups);
    const int tid = threadIdx.x;
    const int col = 4 * (tid % W);
    const int rsub = tid / W;
    const bool colok = col < N;
    int64_t t0 = s * seqlen, t1 = t0 + seqlen;
    if (cu) {
        t0 = min(max((int64_t)cu[s], (int64_t)0), tokens);
        t1 = min(max((int64_t)cu[s + 1], t0), tokens);
    }
    float4 st[kPass];
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
        const int p = i * kRowsPerPass + rsub;
        st[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (init && p < P && colok) st[i] = *reinterpret_cast<const float4*>(init + (sh * P + p) * N + col);
    }
    for (int64_t t = t0; t < t1; ++t) {
        const float a = __expf(gv[t * nheads + h]);
        const float beta = bv[t * nheads + h];
        float kv[4] = {0.f, 0.f, 0.f, 0.f}, qv[4] = {0.f, 0.f, 0.f, 0.f};
        if (colok) {
            const T* kp = Km + (t * ngroups + grp) * N + col;
            const T* qp = Qm + (t * ngroups + grp) * N + col;
#pragma unroll
            for (int e = 0; e < 4; ++e) { kv[e] = to_f32(kp[e]); qv[e] = to_f32(qp[e]); }
        }
        const float kq = group_sum<W>(kv[0] * qv[0] + kv[1] * qv[1] + kv[2] * qv[2] + kv[3] * qv[3]);
        const T* vr = v + (t * nheads + h) * P;
        T* yr = y + (t * nheads + h) * P;
#pragma unroll
        for (int i = 0; i < kPass; ++i) {
            const int p = i * kRowsPerPass + rsub;
            const bool live = p < P;
            float4 c = st[i];
            c.x *= a; c.y *= a; c.z *= a; c.w *= a;
            const float sk = group_sum<W>(c.x * kv[0] + c.y * kv[1] + c.z * kv[2] + c.w * kv[3]);
            const float sq = group_sum<W>(c.x * qv[0] + c.y * qv[1] + c.z * qv[2] + c.w * qv[3]);
            const float u = beta * ((live ? to_f32(vr[p]) : 0.f) - sk);
            st[i] = make_float4(fmaf(u, kv[0], c.x), fmaf(u, kv[1], c.y), fmaf(u, kv[2], c.z), fmaf(u, kv[3], c.w));
            if ((tid % W) == 0 && live) yr[p] = from_f32<T>(fmaf(u, kq, sq));
        }
    }
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
        const int p = i * kRowsPerPass + rsub;
        if (p < P && colok) *reinterpret_cast<float4*>(fin + (sh * P + p) * N + col) = st[i];
    }
}

template <typename T, int W, int P>
hipError_t launch(const T* v, const float* g, const float* beta, const T* k, const T* q, const float* init, T* y,
                  float* fin, const DeltaDims& d, hipStream_t stream)
{
    hipLaunchKernelGGL((delta_fwd_kernel<T, W, P>), dim3((unsigned)(d.seqs * d.nheads)), dim3(256), 0, stream, v, g,
                       beta, k, q, init, y, fin, d.cu, d.seqlen, d.tokens, (int)d.nheads, (int)d.dstate,
                       (int)d.ngroups);
    return hipGetLastError();
}

template <typename T, int W>
hipError_t launch_w(const T* v, const float* g, const float* beta, const T* k, const T* q, const float* init, T* y,
                    float* fin, const DeltaDims& d, hipStream_t stream)
{
    switch (d.headdim) {
    case 16: return launch<T, W, 16>(v, g, beta, k, q, init, y, fin, d, stream);
    case 32: return launch<T, W, 32>(v, g, beta, k, q, init, y, fin, d, stream);
    case 64: return launch<T, W, 64>(v, g, beta, k, q, init, y, fin, d, stream);
    case 128: return launch<T, W, 128>(v, g, beta, k, q, init, y, fin, d, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

size_t delta_forward_workspace(const DeltaDims&, int) { return 256; }

template <typename T>
hipError_t launch_delta_forward(const T* v, const float* g, const float* beta, const T* k, const T* q,
                                const float* init, T* y, float* fin, const DeltaDims& d, void*, hipStream_t stream)
{
    if (d.seqs == 0) return hipSuccess;
    const int64_t w = d.dstate / 4;
    if (w <= 4) return launch_w<T, 4>(v, g, beta, k, q, init, y, fin, d, stream);
    if (w <= 8) return launch_w<T, 8>(v, g, beta, k, q, init, y, fin, d, stream);
    if (w <= 16) return launch_w<T, 16>(v, g, beta, k, q, init, y, fin, d, stream);
    if (w <= 32) return launch_w<T, 32>(v, g, beta, k, q, init, y, fin, d, stream);
    return launch_w<T, 64>(v, g, beta, k, q, init, y, fin, d, stream);
}

template hipError_t launch_delta_forward<float>(const float*, const float*, const float*, const float*, const float*,
                                                const float*, float*, float*, const DeltaDims&, void*, hipStream_t);
template hipError_t launch_delta_forward<bf16>(const bf16*, const float*, const float*, const bf16*, const bf16*,
                                               const float*, bf16*, float*, const DeltaDims&, void*, hipStream_t);

}  // namespace ssd
