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
// where they lead to y only, which is rounded to bf16 itself, S and M are rounded to bf16 once: y is off by 2.4e-3 in
// the 2-norm, of which its own rounding is 1.7e-3. (U is a pair there too, at 2 more matrix instructions a block: 2.8e-3
// without. S as one would cost 8 and 6 % of the time, for 0.1e-3.)
//
// kBwd is the backward's walk forward: the same block by block, in place of y and the final state leaving what the
// walk back and the gradients of k and q need (DeltaKeep). The log decays' gradients need the decayed state's answers
// S' q and S' k to fp32's accuracy of their own (delta_bwd.hip): S' q is y without the token's own update (M below
// its diagonal), S' k = gam K S^T - (A - I) E, neither the difference of larger numbers, on pairs with the low parts'
// product and the third bf16 piece of U and K S^T.
//
// A workgroup = NW wavefronts that walk (16 rows each, of one head or of NH next to each other) and one that feeds
// them: K, Q, the V columns and the blocks' records come through a ring of kBuf stages of asynchronous global -> LDS
// copies, all issued by that one. A wavefront that issues copies stalls while they queue up (28 KB a block at 64
// bytes a cycle), which cost the walk a fifth of its time when its own wavefronts did (192 heads of 64 x 128 over
// 2048 tokens: 74 us against 91, before U was a pair in y; now 79). One barrier per block.
// What bounds it: the chain of one block's products, about 2900 cycles of which a wavefront's matrix instructions
// fill 800 and its vector instructions 900; two wavefronts on a SIMD take 4600 a block. Measured (with U a pair in y):
// 320 heads over 4096 tokens 245 us, 192 over 2048 79, 80 of 64 x 256 over 65536 3490.
#include <type_traits>

#include "delta_tiles.hpp"

namespace ssd {

namespace {

template <typename T, int NB, int NW, int NH, bool kBwd>
struct ChainCfg {
    using R = DeltaRec<T, kBwd>;
    static constexpr int kCH = NB * 32 * (int)sizeof(T) / 16;      // chunks of a K or Q row
    static constexpr int kCV = 16 * NW * (int)sizeof(T) / 16;      // chunks of a V row
    static constexpr int kK = 0, kQ = DTile<kCH>::kBytes, kV = 2 * DTile<kCH>::kBytes,
                         kR = kV + DTile<kCV>::kBytes;
    static constexpr int kStage = kR + NH * R::kFwdBytes;
    // copies of a stage, each of 1 KB
    static constexpr int kCopies = 2 * DTile<kCH>::kInst + DTile<kCV>::kInst + NH * ((R::kFwdBytes + 1023) / 1024);
    // (a third stage of the largest tiles costs registers, and with them a tenth of the time)
    static constexpr int kBuf = 3 * kStage <= (NW > 4 ? 160 : 80) * 1024 ? 3 : 2;
    static constexpr int kLds = kBuf * kStage;
};

template <typename T, int NB, int NW, int NH, bool kBwd>
__device__ __forceinline__ void chain(
    const T* __restrict__ v, const T* __restrict__ Km, const T* __restrict__ Qm, const float* __restrict__ init,
    const unsigned char* __restrict__ recs, T* __restrict__ y, float* __restrict__ fin, DeltaKeep<T> keep, DeltaDims d,
    int nslice)
{
    using C = ChainCfg<T, NB, NW, NH, kBwd>;
    using R = DeltaRec<T, kBwd>;
    constexpr int kBuf = C::kBuf;
    static_assert(C::kLds <= 160 * 1024, "ring");
    extern __shared__ __attribute__((aligned(1024))) unsigned char ring[];        // C::kLds
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    // An XCD takes neighbouring heads, which share K and Q; but sequences of different lengths are dealt out, so that no
    // XCD is left with the long ones (7 of 64 to 4096 tokens, 80 heads: 244 us against 319; started from the longest
    // 223, but ranking them costs 37 short ones 56 us against 46).
    const int bid = d.cu ? (int)blockIdx.x : xcd_logical_block(blockIdx.x, gridDim.x);
    const int slice = bid % nslice;
    const int h0 = (int)(bid / nslice * (int64_t)NH % d.nheads);       // the workgroup's (first) head
    const int64_t s = bid / nslice * (int64_t)NH / d.nheads;
    const DeltaSeq sq = delta_seq(d, s);
    const int grp = h0 / (int)(d.nheads / d.ngroups);
    const int N = (int)d.dstate, P = (int)d.headdim;
    const int pw = 16 * (NW / NH) * slice;                // the workgroup's first column of v
    const int hw = wave / (NW / NH), h = h0 + hw;         // this wavefront's head
    const int64_t sh = s * d.nheads + h;
    const int pv = pw + 16 * (wave % (NW / NH));          // and first column
    const int nblk = (sq.len + kDC - 1) / kDC;
    const int valid = N * (int)sizeof(T) / 16;

    const unsigned krow = (unsigned)(d.ngroups * N * sizeof(T)), vrow = (unsigned)(d.nheads * P * sizeof(T));
    const T* kbase = Km + (sq.start * d.ngroups + grp) * N;
    const T* qbase = Qm + (sq.start * d.ngroups + grp) * N;
    const T* vbase = v + (sq.start * d.nheads + h0) * P + pw;
    const unsigned char* rbase = recs + (sq.slot * d.nheads + h0) * (int64_t)R::kBytes;
    const unsigned lds0 = lds_addr(&ring[0]);
    const WRows<T, C::kCH> krows(r, g);
    const WCols<T, C::kCH> kcols(r, g);
    const WRows<T, kRecCH<T>> rrows(r, g);

    if (valid < C::kCH) {
        // columns past N are never copied: zero them once, so that the state's rows there stay zero
        for (int i = threadIdx.x; i < kBuf * 32 * C::kCH; i += 64 * (NW + 1)) {
            const int row = (i / C::kCH) % 32, b = i / (32 * C::kCH), c = i % C::kCH;
            if (c >= valid) {
                unsigned char* st = ring + b * C::kStage + WTile<C::kCH>::offset(row, c);
                *reinterpret_cast<uint4*>(st + C::kK) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(st + C::kQ) = make_uint4(0, 0, 0, 0);
            }
        }
        __syncthreads();
    }

    if (wave == NW) {
        // the feeding wavefront
        DTileCopy<C::kCH, 1, WTile<C::kCH>> kcopy;
        DTileCopy<C::kCV, 1, VTile<C::kCV>> vcopy;
        kcopy.plan(krow, 0, lane);
        vcopy.plan(vrow, 0, lane);
        auto issue = [&](int c) __attribute__((always_inline)) {
            const unsigned st = lds0 + (unsigned)(c % kBuf) * C::kStage;
            const int rows = sq.len - c * kDC;
            const uint64_t tok = (uint64_t)c * kDC;
            kcopy.issue(reinterpret_cast<const unsigned char*>(kbase) + tok * krow, krow, rows, valid, st + C::kK, 0, lane);
            kcopy.issue(reinterpret_cast<const unsigned char*>(qbase) + tok * krow, krow, rows, valid, st + C::kQ, 0, lane);
            vcopy.issue(reinterpret_cast<const unsigned char*>(vbase) + tok * vrow, vrow, rows, C::kCV, st + C::kV, 0, lane);
#pragma unroll
            for (int i = 0; i < NH; ++i)
                linear_copy<R::kFwdBytes, 1>(rbase + ((int64_t)c * d.nheads + i) * R::kBytes, st + C::kR + i * R::kFwdBytes, 0, lane);
        };
        for (int c = 0; c < kBuf - 1 && c < nblk; ++c) issue(c);
        for (int c = 0; c < nblk; ++c) {
            // Stage c is there when no more than the later stages' copies are outstanding (the counter goes down in
            // order). The last block may have fewer (rows past the sequence are written, not copied): with it in
            // flight, everything is waited for.
            constexpr int kLater = (kBuf - 2) * C::kCopies < 63 ? (kBuf - 2) * C::kCopies : 63;
            if (c + kBuf - 1 >= nblk) wait_vmem(); else wait_vmem_below<kLater>();
            __syncthreads();                              // and everybody is done with the stage before it
            if (c + kBuf - 1 < nblk) issue(c + kBuf - 1);
        }
        return;
    }

    // S^T in accumulator tiles: tile t = 2 kb + x, rows 4g + m = columns ncol(t) + m of the state, column r = its row pv + r
    auto ncol = [&](int t) { return 32 * (t >> 1) + 8 * g + 4 * (t & 1); };
    const int64_t srow = (sh * P + pv + r) * N;
    f32x4 S[2 * NB];
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t) {
        S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (init && ncol(t) < N) S[t] = *reinterpret_cast<const f32x4*>(init + srow + ncol(t));
    }
    auto pair_of = [&](Pair<T>& f, const f32x4& a, const f32x4& b) __attribute__((always_inline)) {
        const float sv[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        f.set(sv);
    };
    // the state entering a chunk of 64 tokens (k = 0 ..) and after the last one
    auto keep_state = [&](int k) __attribute__((always_inline)) {
        const int64_t at = keep.state_at((s * (keep.chunks + 1) + k) * d.nheads + h, pv / 16, lane, d);
#pragma unroll
        for (int kb = 0; kb < NB; ++kb) {
            if (32 * kb < N) {
                Pair<T> s;
                pair_of(s, S[2 * kb], S[2 * kb + 1]);
                store8(keep.S + at + kb * keep.kb_stride, s.hi);
                if constexpr (sizeof(T) == 2) store8(keep.Slo + at + kb * keep.kb_stride, s.lo);
            }
        }
    };
    // dy of this lane's tokens and 4 columns in the columns = tokens form, fetched a block ahead
    f32x4 dyv[2], dyn[2];
    auto fetch_dy = [&](int c) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int64_t tok = sq.start + min(c * kDC + perm32(t, r), sq.len - 1);
            const float4 f = load4f(keep.dy + (tok * d.nheads + h) * P + pv + 4 * g);
            dyn[t] = f32x4{f.x, f.y, f.z, f.w};
        }
    };
    // block c in stage b (a constant: the loop is unrolled over the ring)
    auto step = [&](int c, auto stage) __attribute__((always_inline)) {
        constexpr int b = decltype(stage)::value;
        __syncthreads();                                  // the stage is filled
        if constexpr (kBwd) {
            if (c % 2 == 0) keep_state(c / 2);
#pragma unroll
            for (int t = 0; t < 2; ++t) dyv[t] = dyn[t];
            if (c + 1 < nblk) fetch_dy(c + 1);
        }
        const unsigned st = lds0 + b * C::kStage, rec = st + C::kR + hw * R::kFwdBytes, tab = rec + R::kTab;
        const int rows = min(kDC, sq.len - c * kDC);

        // what does not depend on the state first
        Vec8<T> vf;
        Pair<T> am[2], mm[2];
        float gam8[8], del8[8], gt[2];
        vtile_cols<C::kCV>(vf, st + C::kV, wave, r, g);
        tab_rows(gam8, tab, g);
        tab_rows(del8, tab + 128, g);
        const float gl = lds_at<float>(tab + 124);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            load_pair(am[t], rrows, rec + R::kA, t);
            if constexpr (kBwd) load_pair(mm[t], rrows, rec + R::kM, t); else rrows.load(mm[t].hi, rec + R::kM, t, 0);
            gt[t] = lds_at<float>(tab + 4 * perm32(t, r));
        }

        // K S^T (rows tokens, columns p) and S Q^T (rows p, columns tokens)
        f32x4 ks[2], yt[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) ks[t] = yt[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NB; ++kb) {
            Pair<T> p;
            pair_of(p, S[2 * kb], S[2 * kb + 1]);
            S[2 * kb] *= gl;
            S[2 * kb + 1] *= gl;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                Vec8<T> kf, qf;
                krows.load(kf, st + C::kK, t, kb);
                mma_xp(ks[t], kf, p);
                krows.load(qf, st + C::kQ, t, kb);
                if constexpr (kBwd) mma_px(yt[t], p, qf); else mma(yt[t], p.hi, qf);
            }
        }
        // E = V - gam K S^T (zero in rows past the sequence: their V and K are)
        float E[8], e8[8], dU[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) E[i] = vf.get(i) - gam8[i] * ks[i >> 2][i & 3];
        Pair<T> ep, du;
        ep.set(E);
        if constexpr (kBwd) {
            float ks8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) ks8[i] = gam8[i] * ks[i >> 2][i & 3];
            Pair<T> kp;
            kp.set(ks8);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                f32x4 e = {E[4 * t], E[4 * t + 1], E[4 * t + 2], E[4 * t + 3]};
                mma_pp<true>(e, am[t], ep);
#pragma unroll
                for (int m = 0; m < 4; ++m) e8[4 * t + m] = e[m];
                // x = S' k with columns = tokens, the form in which it is kept
                Vec8<T> one;
                unit_frag(one, t, r, g);
                f32x4 xt = {0.f, 0.f, 0.f, 0.f};
                mma_pp<true>(xt, ep, am[t]);
                xt = -xt;
                mma_rest(xt, kp, ks8, one);
                mma_px(xt, kp, one);
                store4(keep.x + keep.frag(sq.slot + c, h, pv / 16, d) + keep.lane(perm32(t, r), g), xt[0], xt[1], xt[2], xt[3]);
            }
        } else {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                f32x4 e = {E[4 * t], E[4 * t + 1], E[4 * t + 2], E[4 * t + 3]};
                mma_pp(e, am[t], ep);
#pragma unroll
                for (int m = 0; m < 4; ++m) e8[4 * t + m] = e[m];
            }
        }
        // U = beta e (the forward's records have beta in M and in del)
        if constexpr (kBwd) {
            float be[8];
            tab_rows(be, tab + 256, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) e8[i] *= be[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) dU[i] = e8[i] * del8[i];
        du.set(dU);
#pragma unroll
        for (int t = 0; t < 2; ++t) yt[t] *= gt[t];
        if constexpr (kBwd) {
            Pair<T> up;
            up.set(e8);
            float dot[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                mma_rest(yt[t], up, e8, mm[t].hi);
                mma_pp<true>(yt[t], up, mm[t]);
                dot[t] = yt[t][0] * dyv[t][0] + yt[t][1] * dyv[t][1] + yt[t][2] * dyv[t][2] + yt[t][3] * dyv[t][3];
            }
            // (32 tokens as 2 x 64 bytes, each twice; what is past the sequence is not read)
            keep.ydy[((pv / 16 * d.seqs + s) * d.nheads + h) * keep.chunks * 64 + c * kDC + perm32(g >> 1, r)] =
                sum_groups(dot[0], dot[1]);
        } else {
            Pair<T> up;
            up.set(e8);
            // rows past the sequence are outside the buffer: dropped
            const auto out = __builtin_amdgcn_make_buffer_rsrc(
                y + ((sq.start + c * kDC) * d.nheads + h) * P + pv, 0,
                (rows - 1) * (int)vrow + 16 * (int)sizeof(T), kBufferDword3);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                mma_px(yt[t], up, mm[t].hi);
                buffer_store4(out, perm32(t, r) * (int)vrow + 4 * g * (int)sizeof(T), 0, yt[t], T());
            }
        }
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            Vec8<T> kf;
            kcols.load(kf, st + C::kK, t & 1, t >> 1);
            mma_xp(S[t], kf, du);
        }
        settle();                                         // S is read behind the loop's branches
    };
    if constexpr (kBwd) {
        if (nblk > 0) fetch_dy(0);
    }
    for (int c = 0; c < nblk; c += kBuf) {
        step(c, std::integral_constant<int, 0>());
        if (c + 1 < nblk) step(c + 1, std::integral_constant<int, 1>());
        if constexpr (kBuf > 2) {
            if (c + 2 < nblk) step(c + 2, std::integral_constant<int, 2>());
        }
    }
    if constexpr (kBwd) {
        keep_state((int)keep.chunks);
    } else {
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t)
            if (ncol(t) < N) *reinterpret_cast<f32x4*>(fin + srow + ncol(t)) = S[t];
    }
}

// With more than 256 registers at hand the compiler keeps S in accumulation registers, from where every scaling of it
// takes two moves: the bf16 kernels are held to two wavefronts per SIMD, and their LDS is sized at the launch, so
// that the compiler does not conclude from it that there is but one. The fp32 ones, whose fragments take
// twice the registers, need the others.
template <typename T, int NB, int NW, int NH, bool kBwd>
__global__ __launch_bounds__(64 * (NW + 1)) __attribute__((amdgpu_waves_per_eu(NW > 4 ? 3 : 2, NW > 4 ? 3 : 2))) void delta_chain_kernel(
    const T* v, const T* Km, const T* Qm, const float* init, const unsigned char* recs, T* y, float* fin,
    DeltaKeep<T> keep, DeltaDims d, int nslice)
{
    chain<T, NB, NW, NH, kBwd>(v, Km, Qm, init, recs, y, fin, keep, d, nslice);
}
template <typename T, int NB, int NW, int NH, bool kBwd>
__global__ __launch_bounds__(64 * (NW + 1)) void delta_chain_f32_kernel(
    const T* v, const T* Km, const T* Qm, const float* init, const unsigned char* recs, T* y, float* fin,
    DeltaKeep<T> keep, DeltaDims d, int nslice)
{
    chain<T, NB, NW, NH, kBwd>(v, Km, Qm, init, recs, y, fin, keep, d, nslice);
}

template <typename T, int NB, int NW, int NH, bool kBwd>
hipError_t launch_chain(const T* v, const T* k, const T* q, const float* init, const unsigned char* rec, T* y,
                        float* fin, const DeltaKeep<T>& keep, const DeltaDims& d, hipStream_t stream)
{
    const int nslice = (int)d.headdim * NH / (16 * NW);
    const int64_t nblocks = d.seqs * (d.nheads / NH) * nslice;
    if (nblocks == 0) return hipSuccess;
    using C = ChainCfg<T, NB, NW, NH, kBwd>;
    constexpr unsigned kLds = C::kLds;
    if constexpr (sizeof(T) == 2)
        hipLaunchKernelGGL((delta_chain_kernel<T, NB, NW, NH, kBwd>), dim3((unsigned)nblocks), dim3(64 * (NW + 1)), kLds,
                           stream, v, k, q, init, rec, y, fin, keep, d, nslice);
    else
        hipLaunchKernelGGL((delta_chain_f32_kernel<T, NB, NW, NH, kBwd>), dim3((unsigned)nblocks), dim3(64 * (NW + 1)), kLds,
                           stream, v, k, q, init, rec, y, fin, keep, d, nslice);
    return hipGetLastError();
}

template <typename T, int NB, bool kBwd>
hipError_t launch_nw(const T* v, const T* k, const T* q, const float* init, const unsigned char* rec, T* y,
                     float* fin, const DeltaKeep<T>& keep, const DeltaDims& d, hipStream_t stream)
{
#define SSD_CHAIN(NW, NH) return launch_chain<T, NB, NW, NH, kBwd>(v, k, q, init, rec, y, fin, keep, d, stream)
    if constexpr (sizeof(T) == 2 && NB <= 4) {
        // More workgroups of 64 columns than CUs, and a second one does not fit a CU beside the first (its five
        // wavefronts would put four on one SIMD): eight wavefronts that share K and Q, two heads of 64 columns or one
        // of 128. Whole calls, records included: 320 heads of 64 x 128 over 4096 tokens 298 us against 345 with four
        // (their backward 1913 against 2070); 7 sequences of 64 to 4096 tokens, 80 heads, 288 against 314; 37 of 1 to
        // 150, 16 heads of 128 x 128, 51 against 58. With fewer, four: 192 heads over 2048 tokens 104 against 143 with
        // eight, their backward 614 against 692.
        constexpr int64_t kCUs = 256;
        if (d.seqs * d.nheads * d.headdim > 64 * kCUs) {
            if (d.headdim == 128) SSD_CHAIN(8, 1);
            if (d.headdim == 64 && d.nheads / d.ngroups % 2 == 0) SSD_CHAIN(8, 2);
        }
    }
    if (d.headdim == 16) SSD_CHAIN(1, 1);
    // two stages of the widest fp32 rows leave room for two wavefronts' columns
    if (d.headdim == 32 || sizeof(T) * NB == 32) SSD_CHAIN(2, 1);
    if constexpr (sizeof(T) * NB < 32) SSD_CHAIN(4, 1);
#undef SSD_CHAIN
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
