// delta_fwd.hip - the gated delta rule over whole sequences: the walk over the blocks of 32 tokens.
//
// The rows of the state (head-dimension columns p of v) do not mix, so a wavefront takes 16 of them and keeps
// its 16 x N piece of the fp32 state in registers for the whole sequence, transposed: accumulator tiles with rows
// n and columns p.  Two such tiles are an operand fragment as they are (contraction over n), and E, U come out
// of their products in the same form (rows = tokens, columns p), so a block needs no exchange between
// lanes or wavefronts:
//
//   K S^T (rows tokens, columns p) -> E -> e = A E -> U;   Y^T = (S Q^T) diag(gam) + U^T M^T (rows p, columns tokens)
//   S^T = gam_last S^T + K^T (diag(del) U)
//
// For bf16 inputs S, A, E and del U are pairs of bf16 values where they lead to the state (fp32 to about 2^-17);
// where they lead to y only, which is rounded to bf16 itself, S and U are rounded to bf16 once.
//
// kBwd is the backward's walk forward: the same block by block, with y kept to fp32's accuracy (pairs there too)
// and, in place of y and the final state, what the walk back and the gradients of k and q need (DeltaKeep).
//
// A workgroup = NW wavefronts = 16 NW rows of one (sequence, head).  K, Q, the V columns and the block's record come
// through a ring of NBUF stages of asynchronous global -> LDS copies; one barrier per block.
#include "delta_tiles.hpp"

namespace ssd {

namespace {

template <typename T, int NB, int NW, bool kBwd>
struct ChainCfg {
    using R = DeltaRec<T, kBwd>;
    static constexpr int kCH = NB * 32 * (int)sizeof(T) / 16;      // chunks of a K or Q row
    static constexpr int kCV = 16 * NW * (int)sizeof(T) / 16;      // chunks of a V row
    static constexpr int kK = 0, kQ = DTile<kCH>::kBytes, kV = 2 * DTile<kCH>::kBytes,
                         kR = kV + DTile<kCV>::kBytes;
    static constexpr int kStage = kR + R::kFwdBytes;
    static constexpr int kRecInst = (R::kFwdBytes + 1023) / 1024;
    // copies every wavefront makes per stage, at least
    static constexpr int kMin = 2 * (DTile<kCH>::kInst / NW) + DTile<kCV>::kInst / NW + kRecInst / NW;
    static constexpr int kBuf = 3 * kStage <= 80 * 1024 ? 3 : 2 * kStage <= 160 * 1024 ? 2 : 1;
};

template <typename T, int NB, int NW, bool kBwd>
__global__ __launch_bounds__(64 * NW) void delta_chain_kernel(
    const T* __restrict__ v, const T* __restrict__ Km, const T* __restrict__ Qm, const float* __restrict__ init,
    const unsigned char* __restrict__ recs, T* __restrict__ y, float* __restrict__ fin, DeltaKeep<T> keep, DeltaDims d,
    int nslice)
{
    using C = ChainCfg<T, NB, NW, kBwd>;
    using R = DeltaRec<T, kBwd>;
    constexpr int kBuf = C::kBuf;
    static_assert(kBuf >= 2 && kBuf * C::kStage <= 160 * 1024, "ring");
    __shared__ __attribute__((aligned(1024))) unsigned char ring[kBuf * C::kStage];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int bid = xcd_logical_block(blockIdx.x, gridDim.x);
    const int slice = bid % nslice;
    const int64_t sh = bid / nslice;
    const int h = (int)(sh % d.nheads);
    const DeltaSeq sq = delta_seq(d, sh / d.nheads);
    const int grp = h / (int)(d.nheads / d.ngroups);
    const int N = (int)d.dstate, P = (int)d.headdim;
    const int pw = 16 * NW * slice;                       // the workgroup's first column of v
    const int p = pw + 16 * wave + r;                     // this lane's column
    const int nblk = (sq.len + kDC - 1) / kDC;
    const int valid = N * (int)sizeof(T) / 16;

    const unsigned krow = (unsigned)(d.ngroups * N * sizeof(T)), vrow = (unsigned)(d.nheads * P * sizeof(T));
    const T* kbase = Km + (sq.start * d.ngroups + grp) * N;
    const T* qbase = Qm + (sq.start * d.ngroups + grp) * N;
    const T* vbase = v + (sq.start * d.nheads + h) * P + pw;
    T* ybase = y + (sq.start * d.nheads + h) * P + pw + 16 * wave;
    const unsigned char* rbase = recs + (sq.slot * d.nheads + h) * (int64_t)R::kBytes;
    const unsigned lds0 = lds_addr(&ring[0]);

    if (valid < C::kCH) {
        // columns past N are never copied: zero them once, so that the state's rows there stay zero
        for (int i = threadIdx.x; i < kBuf * 32 * C::kCH; i += 64 * NW) {
            const int row = (i / C::kCH) % 32, b = i / (32 * C::kCH), c = i % C::kCH;
            if (c >= valid) {
                unsigned char* st = ring + b * C::kStage + DTile<C::kCH>::offset(row, c);
                *reinterpret_cast<uint4*>(st + C::kK) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(st + C::kQ) = make_uint4(0, 0, 0, 0);
            }
        }
        __syncthreads();
    }

    auto issue = [&](int c) {
        const unsigned st = lds0 + (unsigned)(c % kBuf) * C::kStage;
        const int rmax = min(kDC, sq.len - c * kDC) - 1;
        const int64_t tok = (int64_t)c * kDC;
        dtile_copy<C::kCH, NW>(reinterpret_cast<const unsigned char*>(kbase) + tok * krow, krow, rmax, valid,
                               st + C::kK, wave, lane);
        dtile_copy<C::kCH, NW>(reinterpret_cast<const unsigned char*>(qbase) + tok * krow, krow, rmax, valid,
                               st + C::kQ, wave, lane);
        dtile_copy<C::kCV, NW>(reinterpret_cast<const unsigned char*>(vbase) + tok * vrow, vrow, rmax, C::kCV,
                               st + C::kV, wave, lane);
        linear_copy<R::kFwdBytes, NW>(rbase + (int64_t)c * d.nheads * R::kBytes, st + C::kR, wave, lane);
    };

    f32x4 S[2 * NB];
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t) {
        S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (init && 16 * t < N) {
            const float4 a = *reinterpret_cast<const float4*>(init + (sh * P + p) * N + 16 * t + 4 * g);
            S[t] = f32x4{a.x, a.y, a.z, a.w};
        }
    }
    wait_vmem();          // so that no register load is in flight among the copies that are counted below
#pragma unroll
    for (int c = 0; c < kBuf - 1; ++c)
        if (c < nblk) issue(c);

    // the state entering a chunk of 64 tokens (k = 0 ..) and after the last one
    auto keep_state = [&](int k) {
        const int64_t at = (((sh / d.nheads) * (keep.chunks + 1) + k) * d.nheads + h) * (int64_t)P * N + (int64_t)p * N;
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            if (16 * t < N) {
                store4(keep.S + at + 16 * t + 4 * g, S[t][0], S[t][1], S[t][2], S[t][3]);
                if (sizeof(T) == 2) {
                    float lo[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) lo[m] = S[t][m] - to_f32(from_f32<T>(S[t][m]));
                    store4(keep.Slo + at + 16 * t + 4 * g, lo[0], lo[1], lo[2], lo[3]);
                }
            }
        }
    };

    for (int c = 0; c < nblk; ++c) {
        // this stage's copies are done when no more than the later stages' are outstanding
        constexpr int kLater = (kBuf - 2) * C::kMin < 63 ? (kBuf - 2) * C::kMin : 63;
        if (c + kBuf - 2 < nblk) wait_vmem_below<kLater>(); else wait_vmem();
        __syncthreads();                                  // and everybody is done with the stage before it
        float4 dyv[2];
        if constexpr (kBwd) {
            if (c % 2 == 0) keep_state(c / 2);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int64_t tok = sq.start + min(c * kDC + 16 * t + r, sq.len - 1);
                dyv[t] = load4f(keep.dy + (tok * d.nheads + h) * P + pw + 16 * wave + 4 * g);
            }
        }
        if (c + kBuf - 1 < nblk) issue(c + kBuf - 1);
        const unsigned char* st = ring + (c % kBuf) * C::kStage;
        const unsigned char* rec = st + C::kR;
        const float* tab = reinterpret_cast<const float*>(rec + R::kTab);
        const int rows = min(kDC, sq.len - c * kDC);

        f32x4 ks[2], yt[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) ks[t] = yt[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NB; ++kb) {
            Pair<T> s;
            const float sv[8] = {S[2 * kb][0], S[2 * kb][1], S[2 * kb][2], S[2 * kb][3],
                                 S[2 * kb + 1][0], S[2 * kb + 1][1], S[2 * kb + 1][2], S[2 * kb + 1][3]};
            s.set(sv);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                Vec8<T> kf, qf;
                dtile_row<C::kCH>(kf, st + C::kK, 16 * t + r, kb, g);
                mma_xp(ks[t], kf, s);
                dtile_row<C::kCH>(qf, st + C::kQ, 16 * t + r, kb, g);
                if constexpr (kBwd) mma_px(yt[t], s, qf); else mma(yt[t], s.hi, qf);
            }
        }
        // E = V - gam K S^T, rows past the sequence zero (their copies repeat the last row)
        float E[8];
        {
            Vec8<T> vf;
            dtile_col<C::kCV>(vf, st + C::kV, 16 * wave, r, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int row = (i & 3) + 4 * g + (i >> 2) * 16;
                E[i] = vf.get(i) - tab[row] * ks[i >> 2][i & 3];
            }
            if (rows < kDC) {
#pragma unroll
                for (int i = 0; i < 8; ++i) E[i] = (i & 3) + 4 * g + (i >> 2) * 16 < rows ? E[i] : 0.f;
            }
        }
        Pair<T> ep;
        ep.set(E);
        float U[8], dU[8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            Pair<T> a;
            rec_rows(a, rec + R::kA, t, r, g);
            f32x4 e = {0.f, 0.f, 0.f, 0.f};
            mma_pp(e, a, ep);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int row = 16 * t + 4 * g + m;
                U[4 * t + m] = e[m] * tab[64 + row];
                dU[4 * t + m] = U[4 * t + m] * tab[32 + row];
            }
            if constexpr (kBwd) {
                // e once more with columns = tokens, the form in which it is kept
                f32x4 et = {0.f, 0.f, 0.f, 0.f};
                mma_pp(et, ep, a);
                store4(keep.e + keep.frag(sq.slot + c, h, pw / 16 + wave, d) + t * 256 + lane * 4, et[0], et[1], et[2], et[3]);
            }
        }
        Pair<T> du;
        du.set(dU);
#pragma unroll
        for (int t = 0; t < 2; ++t) yt[t] *= tab[16 * t + r];
        if constexpr (kBwd) {
            Pair<T> up;
            up.set(U);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                Pair<T> m;
                rec_rows(m, rec + R::kM, t, r, g);
                mma_pp(yt[t], up, m);
                float dot = yt[t][0] * dyv[t].x + yt[t][1] * dyv[t].y + yt[t][2] * dyv[t].z + yt[t][3] * dyv[t].w;
                dot += __shfl_xor(dot, 16, kWave);
                dot += __shfl_xor(dot, 32, kWave);
                if (g == 0 && 16 * t + r < rows)
                    keep.ydy[(pw / 16 + wave) * d.tokens * d.nheads + (sq.start + c * kDC + 16 * t + r) * d.nheads + h] = dot;
            }
        } else {
            Vec8<T> uf;
            pack8(uf, U);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                Vec8<T> m;
                dtile_row<kRecCH<T>>(m, rec + R::kM, 16 * t + r, 0, g);
                mma(yt[t], uf, m);
                if (16 * t + r < rows)
                    store4(ybase + (int64_t)(c * kDC + 16 * t + r) * d.nheads * P + 4 * g, yt[t][0], yt[t][1],
                           yt[t][2], yt[t][3]);
            }
        }
        const float gl = tab[31];
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            S[t] *= gl;
            Vec8<T> kf;
            dtile_col<C::kCH>(kf, st + C::kK, 16 * t, r, g);
            mma_xp(S[t], kf, du);
        }
    }
    if constexpr (kBwd) {
        keep_state((int)keep.chunks);
    } else {
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t)
            if (16 * t < N) store4(fin + (sh * P + p) * N + 16 * t + 4 * g, S[t][0], S[t][1], S[t][2], S[t][3]);
    }
}

template <typename T, int NB, int NW, bool kBwd>
hipError_t launch_chain(const T* v, const T* k, const T* q, const float* init, const unsigned char* rec, T* y,
                        float* fin, const DeltaKeep<T>& keep, const DeltaDims& d, hipStream_t stream)
{
    const int nslice = (int)d.headdim / (16 * NW);
    const int64_t nblocks = d.seqs * d.nheads * nslice;
    if (nblocks == 0) return hipSuccess;
    hipLaunchKernelGGL((delta_chain_kernel<T, NB, NW, kBwd>), dim3((unsigned)nblocks), dim3(64 * NW), 0, stream, v, k,
                       q, init, rec, y, fin, keep, d, nslice);
    return hipGetLastError();
}

template <typename T, int NB, bool kBwd>
hipError_t launch_nw(const T* v, const T* k, const T* q, const float* init, const unsigned char* rec, T* y,
                     float* fin, const DeltaKeep<T>& keep, const DeltaDims& d, hipStream_t stream)
{
    if (d.headdim == 16) return launch_chain<T, NB, 1, kBwd>(v, k, q, init, rec, y, fin, keep, d, stream);
    // two stages of the widest fp32 rows leave room for two wavefronts' columns
    if (d.headdim == 32 || sizeof(T) * NB == 32)
        return launch_chain<T, NB, 2, kBwd>(v, k, q, init, rec, y, fin, keep, d, stream);
    if constexpr (sizeof(T) * NB < 32) return launch_chain<T, NB, 4, kBwd>(v, k, q, init, rec, y, fin, keep, d, stream);
    return hipErrorInvalidValue;
}

}  // namespace

size_t delta_forward_workspace(const DeltaDims& d, int elem_bytes)
{
    const size_t rec = elem_bytes == 2 ? DeltaRec<bf16, false>::kBytes : DeltaRec<float, false>::kBytes;
    return ((size_t)(delta_slots(d) * d.nheads) * rec + 255) / 256 * 256 + 256;
}

template <typename T, bool kBwd>
hipError_t launch_delta_chain(const T* v, const T* k, const T* q, const float* init, const unsigned char* rec, T* y,
                              float* fin, const DeltaKeep<T>& keep, const DeltaDims& d, hipStream_t stream)
{
    if (d.dstate <= 32) return launch_nw<T, 1, kBwd>(v, k, q, init, rec, y, fin, keep, d, stream);
    if (d.dstate <= 64) return launch_nw<T, 2, kBwd>(v, k, q, init, rec, y, fin, keep, d, stream);
    if (d.dstate <= 128) return launch_nw<T, 4, kBwd>(v, k, q, init, rec, y, fin, keep, d, stream);
    return launch_nw<T, 8, kBwd>(v, k, q, init, rec, y, fin, keep, d, stream);
}

template <typename T>
hipError_t launch_delta_forward(const T* v, const float* g, const float* beta, const T* k, const T* q,
                                const float* init, T* y, float* fin, const DeltaDims& d, void* workspace,
                                hipStream_t stream)
{
    unsigned char* rec = static_cast<unsigned char*>(workspace);
    hipError_t e = launch_delta_prep<T, false>(k, q, g, beta, rec, d, stream);
    if (e != hipSuccess) return e;
    return launch_delta_chain<T, false>(v, k, q, init, rec, y, fin, DeltaKeep<T>{}, d, stream);
}

#define SSD_DELTA_FWD(T)                                                                                             \
    template hipError_t launch_delta_forward<T>(const T*, const float*, const float*, const T*, const T*,            \
                                                const float*, T*, float*, const DeltaDims&, void*, hipStream_t);     \
    template hipError_t launch_delta_chain<T, true>(const T*, const T*, const T*, const float*,                      \
                                                    const unsigned char*, T*, float*, const DeltaKeep<T>&,           \
                                                    const DeltaDims&, hipStream_t);
SSD_DELTA_FWD(float)
SSD_DELTA_FWD(bf16)
#undef SSD_DELTA_FWD

}  // namespace ssd
