// delta_bwd.hip - gradients of the gated delta rule.
//
// With H = dL/dS after a block of 32 tokens (notation of delta_tiles.hpp; B = (I + diag(beta) X)^-1):
//
//   dU = M^T dY + diag(del) K H^T       w = B^T dU        dV = diag(beta) w       dbeta_i = w_i . e_i
//   dL/dS before = gam_last H + dY^T diag(gam) Q - w^T diag(beta gam) K
//   W = (dY U^T) o G (j <= i)           Z = -(w U^T) o diag(beta) G (j < i)
//   dQ = diag(gam) dY S + W K           dK = W^T Q + (Z + Z^T) K + diag(del) U H - diag(beta gam) w S
//
// and for the log decay, whose gradient is <dL/dS'_t, S'_t>,
//
//   dg_t = dg_{t+1} + l_t,   l_t = dy_t . (S'_t q_t) - dv_t . (S'_t k_t) - u_t . (D_t k_t),   D_t = dL/dS_t without y_t's part
//
// (after a block's last token dg is <H, S>), so it needs row sums only, and the inner product of the two states at the
// ends of every 64-token chunk. Every term of l_t is a product of what lies before token t and what lies behind it, so
// a strong decay makes the terms small with the gradient. (The shorter l_t = dy_t . y_t - dv_t . v_t is the same number,
// but its products within the token cancel: with g = -8 throughout, 1e-3 of dg's norm is lost even in fp32.) With S' k = x
// from the walk forward, e = v - x, w' = D k = dU' + (B - I)^T dU, where dU' = dU - diag(q . k) dY, and w = w' +
// diag(q . k) dY: l = dy . (S' q) - beta (w . x + e . w').
//
// The sum from a chunk's end and the sum from its start differ by the errors of the 64 terms and the two inner products.
// dg_t is the mean of both, each weighted with the other's squared terms (the errors go with the terms): a bridge between two
// known ends, and where an end is large and the gradient is not, as at a last token with a strong decay and a
// gradient of the final state, the sum from the other end. Where S' is zero in fp32 (g below -104) dg is 0.
//
// Four steps: the records (delta_prep); the walk forward again (delta_fwd.hip), keeping x, dy . S' q and the state
// at every 64th token; the walk back (below), the same form with H in the state's place; and, for all chunks of 64
// tokens at once, dq and dk, summed over the heads that share them inside a workgroup, in a fixed order.
// Everything that leads to H, dbeta and dg is computed on pairs (fp32's accuracy for bf16 inputs). dq and dk are rounded
// to T themselves. For bf16 U, W and Z are pairs there too: their rounding was most of the error (2.9e-3 of the norm,
// now 1.8e-3 of which dq's own rounding is 1.66e-3; with one key again and again, where the updates cancel, 1.8e-2 and
// now 2.5e-3) and pairs cost 1 % of the time. S, H, w, gam dY, del U and beta gam w are rounded to bf16 once: the last three
// as pairs leave 1.7e-3 for another 1 %, S's low part would be read for 4 %.
//
// What bounds it: the kept states and values, 7.2 GB written and read (counted) at 4 x 4096 tokens, 80 heads of 64 x 128
// (bf16), 1.94 ms in all: records 147 us (0.64 GB), walk forward 633 (1.9 GB, 3.0 TB/s), walk back 739 (2.5 GB, 3.4 TB/s),
// dq and dk 448 (2.0 GB, 4.5 TB/s), their sums 8, dg and dbeta 31. (With l_t from y and v, and U, W, Z rounded once: 1.83,
// of which 145, 613, 733, 403, 8, 26.)
// A chunk of 64 tokens is what dg's accuracy asks for; the walk back copies with its own wavefronts, as one that feeds
// them took 3 % longer when both were measured.
#include <type_traits>

#include "delta_tiles.hpp"

namespace ssd {

namespace {

constexpr int kChunk = 64;       // tokens of a chunk of the dq, dk step

// What the walk back keeps, beside DeltaKeep.
template <typename T> struct DeltaBack {
    T* w;                    // as x: w of every block, head and 16 columns
    float* sums;             // (headdim / 16, seqs, nheads, 2, 64 chunks): beta (w . x + e . w') and w . e over 16 columns
    T* H;                    // (seqs, chunks, nheads): dL/d(state after each 64-token chunk), as fragments
    float* hs;               // (headdim / 16, seqs, chunks + 1, nheads): <H, S> over 16 rows at the chunks' ends
};

// ---- the walk back ------------------------------------------------------------------------------------------

template <typename T, int NB, int NW>
struct RevCfg {
    using R = DeltaRec<T, true>;
    static constexpr int kCH = NB * 32 * (int)sizeof(T) / 16, kCV = 16 * NW * (int)sizeof(T) / 16;
    static constexpr int kK = 0, kQ = DTile<kCH>::kBytes, kY = 2 * DTile<kCH>::kBytes, kR = kY + DTile<kCV>::kBytes;
    static constexpr int kStage = kR + R::kRevBytes;
    static constexpr int kBuf = 2;
};

// 4 elements as they lie in memory, and as fp32
__device__ __forceinline__ u32x2 load_raw(const bf16* p) { return *reinterpret_cast<const u32x2*>(p); }
__device__ __forceinline__ u32x4 load_raw(const float* p) { return *reinterpret_cast<const u32x4*>(p); }
__device__ __forceinline__ f32x4 raw_f32(u32x2 v)
{
    const bf16x4 q = __builtin_bit_cast(bf16x4, v);
    return f32x4{(float)q[0], (float)q[1], (float)q[2], (float)q[3]};
}
__device__ __forceinline__ f32x4 raw_f32(u32x4 v) { return __builtin_bit_cast(f32x4, v); }

// The stores before and behind this stay instructions of their own (a wait counts them).
__device__ __forceinline__ void own_store() { asm volatile("" ::: "memory"); }

// Row `row`'s columns c .. c + 3 (c a multiple of 4) of a VTile.
template <typename T, int CH>
__device__ __forceinline__ f32x4 vtile_row4(unsigned tile, int row, int c)
{
    constexpr int kPer = 16 / (int)sizeof(T);
    typedef decltype(load_raw(static_cast<const T*>(nullptr))) Raw;
    return raw_f32(lds_at<Raw>(tile + VTile<CH>::offset(row, c / kPer) + (c % kPer) * (int)sizeof(T)));
}

template <typename T, int NB, int NW>
__device__ __forceinline__ void walk_back(
    const T* __restrict__ v, const T* __restrict__ Km, const T* __restrict__ Qm, const float* __restrict__ dfinal,
    const unsigned char* __restrict__ recs, T* __restrict__ dv, float* __restrict__ dinit, DeltaKeep<T> keep,
    DeltaBack<T> back, DeltaDims d, int nslice)
{
    using C = RevCfg<T, NB, NW>;
    using R = DeltaRec<T, true>;
    constexpr int kBuf = C::kBuf;
    static_assert(kBuf * C::kStage <= 160 * 1024, "ring");
    extern __shared__ __attribute__((aligned(1024))) unsigned char ring[];        // kBuf * C::kStage
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int bid = xcd_logical_block(blockIdx.x, gridDim.x);
    const int slice = bid % nslice;
    const int64_t sh = bid / nslice, s = sh / d.nheads;
    const int h = (int)(sh % d.nheads);
    const DeltaSeq sq = delta_seq(d, s);
    const int grp = h / (int)(d.nheads / d.ngroups);
    const int N = (int)d.dstate, P = (int)d.headdim;
    const int pw = 16 * NW * slice, pt = pw / 16 + wave;
    const int p = 16 * pt + r;
    const int nblk = (sq.len + kDC - 1) / kDC;
    const int valid = N * (int)sizeof(T) / 16;
    const unsigned krow = (unsigned)(d.ngroups * N * sizeof(T)), vrow = (unsigned)(d.nheads * P * sizeof(T));
    const T* kbase = Km + (sq.start * d.ngroups + grp) * N;
    const T* qbase = Qm + (sq.start * d.ngroups + grp) * N;
    const T* ybase = keep.dy + (sq.start * d.nheads + h) * P + pw;
    const unsigned char* rbase = recs + (sq.slot * d.nheads + h) * (int64_t)R::kBytes + R::kM;
    const unsigned lds0 = lds_addr(&ring[0]);
    const WRows<T, C::kCH> krows(r, g);
    const WCols<T, C::kCH> kcols(r, g);
    const WCols<T, kRecCH<T>> rcols(r, g);
    DTileCopy<C::kCH, NW, WTile<C::kCH>> kcopy;
    DTileCopy<C::kCV, NW, VTile<C::kCV>> vcopy;
    kcopy.plan(krow, wave, lane);
    vcopy.plan(vrow, wave, lane);

    if (valid < C::kCH) {
        for (int i = threadIdx.x; i < kBuf * 32 * C::kCH; i += 64 * NW) {
            const int row = (i / C::kCH) % 32, b = i / (32 * C::kCH), c = i % C::kCH;
            if (c >= valid) {
                unsigned char* st = ring + b * C::kStage + WTile<C::kCH>::offset(row, c);
                *reinterpret_cast<uint4*>(st + C::kK) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(st + C::kQ) = make_uint4(0, 0, 0, 0);
            }
        }
        __syncthreads();
    }
    // the copies of block c (called from the last to the first) into stage b
    const int last = nblk > 0 ? nblk - 1 : 0;
    const unsigned char* kp = reinterpret_cast<const unsigned char*>(kbase) + (uint64_t)krow * kDC * last;
    const unsigned char* qp = reinterpret_cast<const unsigned char*>(qbase) + (uint64_t)krow * kDC * last;
    const unsigned char* yp = reinterpret_cast<const unsigned char*>(ybase) + (uint64_t)vrow * kDC * last;
    const unsigned char* rp = rbase + (int64_t)last * d.nheads * R::kBytes;
    auto issue = [&](int c, int b) __attribute__((always_inline)) {
        const unsigned st = lds0 + (unsigned)b * C::kStage;
        const int rows = sq.len - c * kDC;
        kcopy.issue(kp, krow, rows, valid, st + C::kK, wave, lane);
        kcopy.issue(qp, krow, rows, valid, st + C::kQ, wave, lane);
        vcopy.issue(yp, vrow, rows, C::kCV, st + C::kY, wave, lane);
        linear_copy<R::kRevBytes, NW>(rp, st + C::kR, wave, lane);
        kp -= (uint64_t)krow * kDC;
        qp -= (uint64_t)krow * kDC;
        yp -= (uint64_t)vrow * kDC;
        rp -= d.nheads * R::kBytes;
    };

    auto ncol = [&](int t) { return 32 * (t >> 1) + 8 * g + 4 * (t & 1); };        // as in the walk forward
    f32x4 H[2 * NB];
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t) {
        H[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (dfinal && ncol(t) < N) {
            const float4 a = *reinterpret_cast<const float4*>(dfinal + (sh * P + p) * N + ncol(t));
            H[t] = f32x4{a.x, a.y, a.z, a.w};
        }
    }
    // S at the start of chunk k (or the end), as it is kept, for <H, S> over this wavefront's rows. Where registers
    // allow, it is fetched a block ahead.
    constexpr bool kAhead = NB * sizeof(T) <= 8;
    typedef decltype(load_raw(static_cast<const T*>(nullptr))) Raw;
    Vec8<T> shi[kAhead ? NB : 1], slo[kAhead && sizeof(T) == 2 ? NB : 1];
    auto at_S = [&](int k) { return keep.state_at((s * (keep.chunks + 1) + k) * d.nheads + h, pt, lane, d); };
    auto fetch_S = [&](int k) __attribute__((always_inline)) {
        if constexpr (kAhead) {
            const int64_t at = at_S(k);
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                if (32 * kb < N) {
                    load8(shi[kb], keep.S + at + kb * keep.kb_stride);
                    if constexpr (sizeof(T) == 2) load8(slo[kb], keep.Slo + at + kb * keep.kb_stride);
                }
            }
        }
    };
    auto put_inner = [&](int k) __attribute__((always_inline)) {
        const int64_t at = at_S(k);
        float dot = 0.f;
#pragma unroll
        for (int kb = 0; kb < NB; ++kb) {
            if (32 * kb < N) {
                Vec8<T> a, l;
                if constexpr (kAhead) a = shi[kb]; else load8(a, keep.S + at + kb * keep.kb_stride);
                if constexpr (sizeof(T) == 2) {
                    if constexpr (kAhead) l = slo[kb]; else load8(l, keep.Slo + at + kb * keep.kb_stride);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dot = fmaf(H[2 * kb + (i >> 2)][i & 3], a.get(i), dot);
                    if constexpr (sizeof(T) == 2) dot = fmaf(H[2 * kb + (i >> 2)][i & 3], l.get(i), dot);
                }
            }
        }
        dot = group_sum<64>(dot);
        if (lane == 0) back.hs[((pt * d.seqs + s) * (keep.chunks + 1) + k) * d.nheads + h] = dot;
    };
    // v and x of this lane's tokens and 4 columns in the columns = tokens form, fetched a block ahead
    Raw vv[2], vn[2];
    f32x4 xv[2], xn[2];
    auto fetch_vx = [&](int c) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int64_t tok = sq.start + min(c * kDC + perm32(t, r), sq.len - 1);
            vn[t] = load_raw(v + (tok * d.nheads + h) * P + 16 * pt + 4 * g);
            xn[t] = *reinterpret_cast<const f32x4*>(keep.x + keep.frag(sq.slot + c, h, pt, d) + keep.lane(perm32(t, r), g));
        }
    };
    if (nblk > 0) {
        fetch_S((nblk + 1) / 2);
        fetch_vx(nblk - 1);
    } else {
        fetch_S(0);
    }
    wait_vmem();
    if (nblk > 0) issue(nblk - 1, 0);

    auto step = [&](int c, auto stage) __attribute__((always_inline)) {
        constexpr int b = decltype(stage)::value;
        // (see the walk forward; the loads ahead of the next block were started before its copies)
        // Behind the last copy lie this many stores of the block before, each at least one instruction: own_store()
        // stands between those that could become one.
        constexpr int kStores = 5;
        if (c < nblk - 1) wait_vmem_below<kStores>(); else wait_vmem();
        __syncthreads();
        if (c % 2 == 1 || c == nblk - 1) {
            const int k = c / 2;
            const int64_t at = keep.state_at((s * keep.chunks + k) * d.nheads + h, pt, lane, d);
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                if (32 * kb < N) {
                    const float hv[8] = {H[2 * kb][0], H[2 * kb][1], H[2 * kb][2], H[2 * kb][3],
                                         H[2 * kb + 1][0], H[2 * kb + 1][1], H[2 * kb + 1][2], H[2 * kb + 1][3]};
                    Vec8<T> hf;
                    pack8(hf, hv);
                    store8(back.H + at + kb * keep.kb_stride, hf);
                }
            }
            put_inner(k + 1);
        }
        if (c % 2 == 0) fetch_S(c / 2);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            vv[t] = vn[t];
            xv[t] = xn[t];
        }
        if (c > 0) {
            fetch_vx(c - 1);
            issue(c - 1, 1 - b);
        }
        const unsigned st = lds0 + b * C::kStage, rec = st + C::kR - R::kM, tab = rec + R::kTab;
        const int rows = min(kDC, sq.len - c * kDC);

        // what does not depend on H first
        Vec8<T> yf;
        Pair<T> mt[2], bm[2];
        float ga[8], de[8], bt8[8], bet[2];
        vtile_cols<C::kCV>(yf, st + C::kY, wave, r, g);
        tab_rows(ga, tab, g);
        tab_rows(de, tab + 128, g);
        tab_rows(bt8, tab + 256, g);
        const float gl = lds_at<float>(tab + 124);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            load_pair(mt[t], rcols, rec + R::kM, t);
            load_pair(bm[t], rcols, rec + R::kB, t);
            bet[t] = lds_at<float>(tab + 256 + 4 * perm32(t, r));
        }

        // dU = M^T dY + del K H^T (rows tokens, columns p; rows past the sequence are zero, as their dY and K are)
        f32x4 kh[2], du[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) kh[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NB; ++kb) {
            Pair<T> hp;
            const float hv[8] = {H[2 * kb][0], H[2 * kb][1], H[2 * kb][2], H[2 * kb][3],
                                 H[2 * kb + 1][0], H[2 * kb + 1][1], H[2 * kb + 1][2], H[2 * kb + 1][3]};
            hp.set(hv);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                Vec8<T> kf;
                krows.load(kf, st + C::kK, t, kb);
                mma_xp(kh[t], kf, hp);
            }
        }
        // dU' is without M's diagonal, dU with it
        float dU[8], dO[8], qk8[8];
        tab_rows(qk8, tab + 384, g);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int m = 0; m < 4; ++m) du[t][m] = kh[t][m] * de[4 * t + m];
            mma_px(du[t], mt[t], yf);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                dO[4 * t + m] = du[t][m];
                dU[4 * t + m] = fmaf(qk8[4 * t + m], yf.get(4 * t + m), du[t][m]);
            }
        }
        Pair<T> dup, dop;
        dup.set(dU);
        dop.set(dO);
        // w = B^T dU in both forms: rows tokens (to go on with) and columns tokens (to hand out). Rows past the
        // sequence are outside the buffers: dropped.
        const int64_t th = (sq.start + c * kDC) * d.nheads + h;
        const auto odv = __builtin_amdgcn_make_buffer_rsrc(dv + th * P + 16 * pt, 0, (rows - 1) * (int)vrow + 16 * (int)sizeof(T), kBufferDword3);
        float we[2], ll[2];
        float bw[8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            Vec8<T> one;
            unit_frag(one, t, r, g);
            f32x4 w = {dU[4 * t], dU[4 * t + 1], dU[4 * t + 2], dU[4 * t + 3]}, wo = {0.f, 0.f, 0.f, 0.f};
            mma_pp<true>(w, bm[t], dup);
            mma_pp<true>(wo, dup, bm[t]);
            mma_rest(wo, dop, dO, one);
            mma_px(wo, dop, one);
            const float qk = lds_at<float>(tab + 384 + 4 * perm32(t, r));
            f32x4 wt = wo + qk * vtile_row4<T, C::kCV>(st + C::kY, perm32(t, r), 16 * wave + 4 * g);
#pragma unroll
            for (int m = 0; m < 4; ++m) bw[4 * t + m] = -ga[4 * t + m] * bt8[4 * t + m] * w[m];
            store4(back.w + keep.frag(sq.slot + c, h, pt, d) + keep.lane(perm32(t, r), g), wt[0], wt[1], wt[2], wt[3]);
            const f32x4 ev = raw_f32(vv[t]) - xv[t];
            we[t] = wt[0] * ev[0] + wt[1] * ev[1] + wt[2] * ev[2] + wt[3] * ev[3];
            ll[t] = bet[t] * (wt[0] * xv[t][0] + wt[1] * xv[t][1] + wt[2] * xv[t][2] + wt[3] * xv[t][3] +
                              wo[0] * ev[0] + wo[1] * ev[1] + wo[2] * ev[2] + wo[3] * ev[3]);
            wt *= bet[t];
            buffer_store4(odv, perm32(t, r) * (int)vrow + 4 * g * (int)sizeof(T), 0, wt, T());
            own_store();
        }
        // lane group g: beta (w . x + e . w') (g even) or w . e of tile g / 2
        back.sums[(((pt * d.seqs + s) * d.nheads + h) * 2 + (g & 1)) * keep.chunks * 64 + c * kDC + perm32(g >> 1, r)] =
            sum_groups(ll[0], ll[1], we[0], we[1]);
        // H before the block = gam_last H + Q^T (gam dY) - K^T (beta gam w)
        float gy[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) gy[i] = ga[i] * yf.get(i);
        Pair<T> gyp, bwp;
        gyp.set(gy);
        bwp.set(bw);
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            H[t] *= gl;
            Vec8<T> qf, kf;
            kcols.load(qf, st + C::kQ, t & 1, t >> 1);
            mma_xp(H[t], qf, gyp);
            kcols.load(kf, st + C::kK, t & 1, t >> 1);
            mma_xp(H[t], kf, bwp);
        }
        settle();                                         // H is read behind the loop's branches
    };
    for (int c = nblk - 1; c >= 0; c -= 2) {
        step(c, std::integral_constant<int, 0>());
        if (c > 0) step(c - 1, std::integral_constant<int, 1>());
    }
    put_inner(0);
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t)
        if (ncol(t) < N) store4(dinit + (sh * P + p) * N + ncol(t), H[t][0], H[t][1], H[t][2], H[t][3]);
}

// (registers: see delta_chain_kernel)
template <typename T, int NB, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2))) void delta_rev_kernel(
    const T* v, const T* Km, const T* Qm, const float* dfinal, const unsigned char* recs, T* dv, float* dinit,
    DeltaKeep<T> keep, DeltaBack<T> back, DeltaDims d, int nslice)
{
    walk_back<T, NB, NW>(v, Km, Qm, dfinal, recs, dv, dinit, keep, back, d, nslice);
}
template <typename T, int NB, int NW>
__global__ __launch_bounds__(64 * NW) void delta_rev_f32_kernel(
    const T* v, const T* Km, const T* Qm, const float* dfinal, const unsigned char* recs, T* dv, float* dinit,
    DeltaKeep<T> keep, DeltaBack<T> back, DeltaDims d, int nslice)
{
    walk_back<T, NB, NW>(v, Km, Qm, dfinal, recs, dv, dinit, keep, back, d, nslice);
}

// ---- dbeta and dg ---------------------------------------------------------------------------------------------

// A wavefront = one 64-token chunk of one head, lane = token; a workgroup = that chunk of 16 heads, whose results are
// turned in LDS so that they leave as pieces of token rows.
__global__ __launch_bounds__(256) void delta_scalar_kernel(
    const float* __restrict__ ydy, const float* __restrict__ sums, const float* __restrict__ hs,
    const float* __restrict__ gv, float* __restrict__ dg, float* __restrict__ dbeta, DeltaDims d, int64_t chunks,
    int hblocks, int zero_first)
{
    __shared__ float og[64][17], ob[64][17];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int h0 = (int)(blockIdx.x % hblocks) * 16;
    const int64_t sk = blockIdx.x / hblocks, s = sk / chunks, k = sk % chunks;
    const int left = (int)min(d.seqlen - 64 * k, (int64_t)64);
    const int npt = (int)d.headdim / 16;
    for (int i = wave; i < 16; i += 4) {
        const int h = h0 + i;
        if (h >= d.nheads) break;
        float b = 0.f;
        // the sums, and in 16 columns each, their squares: what the weights are made of
        double loc = 0.0, loc2 = 0.0, start = 0.0, start2 = 0.0, end = 0.0, end2 = 0.0;
        for (int pt = 0; pt < npt; ++pt) {
            const int64_t row = (pt * d.seqs + s) * d.nheads + h;
            if (lane < left) {
                const float* at = sums + row * 2 * chunks * 64 + k * 64 + lane;
                const double p = ydy[row * chunks * 64 + k * 64 + lane], q = at[0];
                loc += p - q;
                loc2 += (fabs(p) + fabs(q)) * (fabs(p) + fabs(q));
                b += at[chunks * 64];
            }
            const float* e = hs + ((pt * d.seqs + s) * (chunks + 1) + k) * d.nheads + h;
            const double e0 = e[0], e1 = e[d.nheads];
            start += e0;
            start2 += e0 * e0;
            end += e1;
            end2 += e1 * e1;
        }
        // sums from this token to the chunk's end, and from the chunk's start to before it
        double down = loc, down2 = loc2, up = loc, up2 = loc2;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const double a = __shfl_down(down, m, 64), a2 = __shfl_down(down2, m, 64);
            const double c = __shfl_up(up, m, 64), c2 = __shfl_up(up2, m, 64);
            if (lane + m < 64) { down += a; down2 += a2; }
            if (lane >= m) { up += c; up2 += c2; }
        }
        up = __shfl_up(up, 1, 64);
        up2 = __shfl_up(up2, 1, 64);
        const double from_end = end + down, from_start = lane ? start - up : start;
        const double w_start = end2 + down2, w_end = lane ? start2 + up2 : start2;
        og[lane][i] = (float)(w_start + w_end > 0.0 ? (from_start * w_start + from_end * w_end) / (w_start + w_end) : from_end);
        ob[lane][i] = b;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < 1024; j += 256) {
        const int t = j / 16, i = j % 16;
        if (t < left && h0 + i < d.nheads) {
            const int64_t at = (s * d.seqlen + k * 64 + t) * d.nheads + h0 + i;
            // without an initial state nothing decays into the first token, and nothing into one that resets the state
            dg[at] = (zero_first && k == 0 && t == 0) || gv[at] < -104.f ? 0.f : og[t][i];
            dbeta[at] = ob[t][i];
        }
    }
}

// ---- dq and dk ------------------------------------------------------------------------------------------------

template <typename T, int NB>
struct KqCfg {
    static constexpr int kCH = NB * 32 * (int)sizeof(T) / 16;
    static constexpr int kTile = DTile<kCH>::kBytes;               // 32 rows of S, H, K or Q
    static constexpr int kStage = 2 * kTile;
    static constexpr int kCW = kChunk * (int)sizeof(T) / 16;       // chunks of a row of W or Z
    static constexpr int kWz = 2 * DTile<kCW>::kBytes;             // W or Z: 64 rows, a plane
    static constexpr int kPlanes = sizeof(T) == 2 ? 2 : 1;         // of W, Z and U: pairs
    static constexpr int kEpi = 2 * kTile + 2 * kPlanes * kWz;
    static constexpr int kRing = 2 * kStage > kEpi ? 2 * kStage : kEpi;
    static constexpr int kU = kPlanes * 4 * 64 * 8 * (int)sizeof(T);   // U of 64 tokens x 32 columns as fragments
};

// A workgroup = one 64-token chunk of one (row, group) and a range of the group's heads; a wavefront = 16 of the
// tokens and all N columns of dq and dk (as rows n, columns = tokens).
template <typename T, int NB>
__global__ __launch_bounds__(256, 2) void delta_kq_kernel(
    const T* __restrict__ v, const T* __restrict__ Km, const T* __restrict__ Qm, const float* __restrict__ gv,
    const float* __restrict__ bv, DeltaKeep<T> keep, DeltaBack<T> back, T* __restrict__ dq, T* __restrict__ dk, float* __restrict__ partial,
    DeltaDims d, int nslice)
{
    using C = KqCfg<T, NB>;
    __shared__ __attribute__((aligned(1024))) unsigned char ring[C::kRing];
    __shared__ __attribute__((aligned(16))) unsigned char ub[2][C::kU];
    __shared__ double cst[4][64];
    __shared__ float bet[4][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int slice = blockIdx.x % nslice;
    const int grp = (blockIdx.x / nslice) % d.ngroups;
    const int64_t sk = blockIdx.x / nslice / d.ngroups, s = sk / keep.chunks;
    const int k = (int)(sk % keep.chunks);
    const int N = (int)d.dstate, P = (int)d.headdim, L = (int)d.seqlen;
    const int hpg = (int)(d.nheads / d.ngroups);
    const int h0 = grp * hpg + hpg * slice / nslice, h1 = grp * hpg + hpg * (slice + 1) / nslice;
    const int rows = min(kChunk, L - k * kChunk);
    const int nkb = (P + 31) / 32, nst = (h1 - h0) * nkb;
    const int valid = N * (int)sizeof(T) / 16;
    const int64_t t0 = s * d.seqlen + (int64_t)k * kChunk;
    const int nc32 = (L + kDC - 1) / kDC;
    const int64_t slot = s * nc32 + 2 * k + (wave >> 1);
    const bool blk = 2 * k + (wave >> 1) < nc32;              // this wavefront's block of 32 exists
    const int mine = 16 * wave + r;                           // this lane's token in operand fragments
    const bool tok = mine < rows;
    const unsigned lds0 = lds_addr(&ring[0]);
    const DCols<T, C::kCH> cols(r, g);
    // 32 rows of a kept state (two 16-row pieces of fragments) into a tile
    constexpr int kIs = DTile<C::kCH>::kInst, kKs = (kIs + 3) / 4;
    const int nkc = (N + 31) / 32;
    auto copy_state = [&](const T* m, int rows, unsigned lds) __attribute__((always_inline)) {
#pragma unroll
        for (int q4 = 0; q4 < kKs; ++q4) {
            const int q = wave + 4 * q4;
            if (kIs % 4 != 0 && q >= kIs) break;
            int rr, c;
            DTileCopy<C::kCH, 4>::place(q, lane, rr, c);
            // chunk c: 16 / sizeof(T) of the columns 8 gc .. 8 gc + 7 of the 32 numbered kc
            constexpr int kPer = 8 * (int)sizeof(T) / 16;
            const int kc = c / (4 * kPer), gc = c / kPer % 4, part = c % kPer;
            const unsigned off = (unsigned)(((rr >> 4) * nkc + kc) * 512 + (16 * gc + (rr & 15)) * 8) * (unsigned)sizeof(T) + 16u * part;
            if (c < valid) {
                if (rr < rows)
                    dma16_off(m, off, lds + q * 1024u);
                else
                    *(__attribute__((address_space(3))) u32x4*)(uintptr_t)(lds + q * 1024u + lane * 16u) = u32x4{0, 0, 0, 0};
            }
        }
    };

    auto zero_pad = [&](int tiles) {
        for (int i = threadIdx.x; i < tiles * 32 * C::kCH; i += 256) {
            const int c = i % C::kCH;
            if (c >= valid)
                *reinterpret_cast<uint4*>(ring + (i / (32 * C::kCH)) * C::kTile +
                                          DTile<C::kCH>::offset((i / C::kCH) % 32, c)) = make_uint4(0, 0, 0, 0);
        }
    };
    if (valid < C::kCH) {
        zero_pad(4);
        __syncthreads();
    }
    auto issue = [&](int i) __attribute__((always_inline)) {
        const int h = h0 + i / nkb, kb = i % nkb;
        const unsigned st = lds0 + (unsigned)(i & 1) * C::kStage;
        const int rows = P - 32 * kb;
        const int64_t off = (int64_t)2 * kb * nkc * 512;
        copy_state(keep.S + ((s * (keep.chunks + 1) + k) * d.nheads + h) * keep.plane(d) + off, rows, st);
        copy_state(back.H + ((s * keep.chunks + k) * d.nheads + h) * keep.plane(d) + off, rows, st + C::kTile);
    };
    // the operands of a stage in registers: lane = token, slots = columns {4g .., 16 + 4g ..} of 32
    typedef decltype(load_raw(static_cast<const T*>(nullptr))) Raw;
    struct Ops { float4 y[2], x[2], w[2]; Raw v[2]; float gr, be; };
    auto fetch = [&](int i) __attribute__((always_inline)) {
        Ops o;
        const int h = h0 + i / nkb, kb = i % nkb;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            o.y[t] = o.x[t] = o.w[t] = make_float4(0.f, 0.f, 0.f, 0.f);
            o.v[t] = Raw{};
            if (tok && blk && 32 * kb + 16 * t < P) {
                const int64_t at = ((t0 + mine) * d.nheads + h) * P + 32 * kb + 16 * t + 4 * g;
                o.y[t] = load4f(keep.dy + at);
                o.v[t] = load_raw(v + at);
                const int64_t f = keep.frag(slot, h, 2 * kb + t, d) + (wave & 1) * 256 + lane * 4;
                o.x[t] = load4f(keep.x + f);
                o.w[t] = load4f(back.w + f);
            }
        }
        const int64_t at = (t0 + min(lane, rows - 1)) * d.nheads + h;
        o.gr = gv[at];
        o.be = bv[at];
        return o;
    };

    f32x4 aq[2 * NB], ak[2 * NB], Ws[4], Zs[4], wa[4], za[4];
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t) aq[t] = ak[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 4; ++t) Ws[t] = Zs[t] = wa[t] = za[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    issue(0);
    Ops cur = fetch(0);
    for (int i = 0; i < nst; ++i) {
        const int kb = i % nkb;
        if (kb == 0) {
            // the head's decays: every wavefront sums the 64 tokens' for itself, lane = token
            double cs = lane < rows ? (double)(cur.gr < -1000.f ? -1000.f : cur.gr) : 0.0;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const double up = __shfl_up(cs, m, kWave);
                if (lane >= m) cs += up;
            }
            cst[wave][lane] = cs;
            bet[wave][lane] = lane < rows ? cur.be : 0.f;
        }
        const double ci = cst[wave][mine];
        const float gam = __expf((float)ci), del = __expf((float)(cst[wave][63] - ci)), be = bet[wave][mine];
        float f[8];
        const float yv[8] = {cur.y[0].x, cur.y[0].y, cur.y[0].z, cur.y[0].w, cur.y[1].x, cur.y[1].y, cur.y[1].z, cur.y[1].w};
        const float xv[8] = {cur.x[0].x, cur.x[0].y, cur.x[0].z, cur.x[0].w, cur.x[1].x, cur.x[1].y, cur.x[1].z, cur.x[1].w};
        const f32x4 v0 = raw_f32(cur.v[0]), v1 = raw_f32(cur.v[1]);
        const float ev[8] = {v0[0] - xv[0], v0[1] - xv[1], v0[2] - xv[2], v0[3] - xv[3],
                             v1[0] - xv[4], v1[1] - xv[5], v1[2] - xv[6], v1[3] - xv[7]};
        const float wv[8] = {cur.w[0].x, cur.w[0].y, cur.w[0].z, cur.w[0].w, cur.w[1].x, cur.w[1].y, cur.w[1].z, cur.w[1].w};
        Vec8<T> yf, wf, gy, du, bw, uf;
        pack8(yf, yv);
        pack8(wf, wv);
#pragma unroll
        for (int m = 0; m < 8; ++m) f[m] = gam * yv[m];
        pack8(gy, f);
#pragma unroll
        for (int m = 0; m < 8; ++m) f[m] = be * ev[m];
        Pair<T> up;
        up.set(f);
#pragma unroll
        for (int m = 0; m < 8; ++m) f[m] *= del;
        pack8(du, f);
#pragma unroll
        for (int m = 0; m < 8; ++m) f[m] = -be * gam * wv[m];
        pack8(bw, f);
        T* un = reinterpret_cast<T*>(ub[i & 1]) + (wave * 64 + lane) * 8;
        store8(un, up.hi);
        if constexpr (sizeof(T) == 2) store8(un + 4 * 64 * 8, up.lo);
        wait_vmem();
        __syncthreads();
        if (i + 1 < nst) {
            issue(i + 1);
            cur = fetch(i + 1);
        }
        const unsigned st = lds0 + (unsigned)(i & 1) * C::kStage;
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            Vec8<T> sf, hf;
            cols.load(sf, st, t);
            cols.load(hf, st + C::kTile, t);
            mma(aq[t], sf, gy);
            mma(ak[t], hf, du);
            mma(ak[t], sf, bw);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t <= wave) {
                Pair<T> u;
                load8(u.hi, reinterpret_cast<const T*>(ub[i & 1]) + (t * 64 + lane) * 8);
                if constexpr (sizeof(T) == 2) load8(u.lo, reinterpret_cast<const T*>(ub[i & 1]) + 4 * 64 * 8 + (t * 64 + lane) * 8);
                mma_xp(wa[t], yf, u);
                mma_xp(za[t], wf, u);
            }
        }
        settle();
        if (kb == nkb - 1) {
            // the head's W and Z, rows i = 16 wave + 4g + m, columns j = 16 t + r
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (t <= wave) {
                    const double cj = cst[wave][16 * t + r];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const int ri = 16 * wave + 4 * g + m, rj = 16 * t + r;
                        const float G = rj <= ri ? __expf((float)(cst[wave][ri] - cj)) : 0.f;
                        Ws[t][m] = fmaf(G, wa[t][m], Ws[t][m]);
                        Zs[t][m] = fmaf(rj < ri ? -G * bet[wave][ri] : 0.f, za[t][m], Zs[t][m]);
                    }
                    wa[t] = za[t] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
            }
        }
    }
    __syncthreads();
    // W and Z to LDS behind the place of K's two tiles (whose pad columns are zero still): dq += W K, dk += (Z + Z^T) K, then Q in K's place: dk += W^T Q
    unsigned char* const wl = ring + 2 * C::kTile;
    unsigned char* const zl = wl + C::kPlanes * C::kWz;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int row = 16 * (wave & 1) + 4 * g + m, col = 16 * t + r;
            constexpr int kPer = 16 / (int)sizeof(T);
            const int o = (wave >> 1) * DTile<C::kCW>::kBytes + DTile<C::kCW>::offset(row, col / kPer) +
                          (col % kPer) * (int)sizeof(T);
            const T wh = from_f32<T>(Ws[t][m]), zh = from_f32<T>(Zs[t][m]);
            *reinterpret_cast<T*>(wl + o) = wh;
            *reinterpret_cast<T*>(zl + o) = zh;
            if constexpr (C::kPlanes == 2) {
                *reinterpret_cast<T*>(wl + C::kWz + o) = from_f32<T>(Ws[t][m] - to_f32(wh));
                *reinterpret_cast<T*>(zl + C::kWz + o) = from_f32<T>(Zs[t][m] - to_f32(zh));
            }
        }
    }
    DTileCopy<C::kCH, 4> kcopy;
    kcopy.plan((unsigned)(d.ngroups * N * sizeof(T)), wave, lane);
    auto load_rows = [&](const T* m) __attribute__((always_inline)) {
        for (int b = 0; b < 2; ++b) {
            kcopy.issue(m + ((t0 + 32 * b) * d.ngroups + grp) * N, (unsigned)(d.ngroups * N * sizeof(T)), rows - 32 * b,
                        valid, lds0 + b * C::kTile, wave, lane);
        }
        wait_vmem();
        __syncthreads();
    };
    const unsigned wl0 = lds0 + 2 * C::kTile;
    const DRows<T, C::kCW> wrows(r, g);
    load_rows(Km);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const unsigned wt = wl0 + (wave >> 1) * DTile<C::kCW>::kBytes, zt = wt + C::kPlanes * C::kWz;
        const unsigned ct = wl0 + C::kPlanes * C::kWz + b * DTile<C::kCW>::kBytes;
        Pair<T> wr, zr, zc;
        wrows.load(wr.hi, wt, wave & 1, b);
        wrows.load(zr.hi, zt, wave & 1, b);
        DCols<T, C::kCW>::load_any(zc.hi, ct, wave, r, g);
        if constexpr (C::kPlanes == 2) {
            wrows.load(wr.lo, wt + C::kWz, wave & 1, b);
            wrows.load(zr.lo, zt + C::kWz, wave & 1, b);
            DCols<T, C::kCW>::load_any(zc.lo, ct + C::kWz, wave, r, g);
        }
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            Vec8<T> kf;
            cols.load(kf, lds0 + b * C::kTile, t);
            mma_xp(aq[t], kf, wr);
            mma_xp(ak[t], kf, zr);
            mma_xp(ak[t], kf, zc);
        }
    }
    __syncthreads();
    load_rows(Qm);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        Pair<T> wc;
        DCols<T, C::kCW>::load_any(wc.hi, wl0 + b * DTile<C::kCW>::kBytes, wave, r, g);
        if constexpr (C::kPlanes == 2) DCols<T, C::kCW>::load_any(wc.lo, wl0 + C::kWz + b * DTile<C::kCW>::kBytes, wave, r, g);
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            Vec8<T> qf;
            cols.load(qf, lds0 + b * C::kTile, t);
            mma_xp(ak[t], qf, wc);
        }
    }
    settle();
    if (!tok) return;
    const int64_t at = ((t0 + mine) * d.ngroups + grp) * N + 4 * g;
    const int64_t all = d.tokens * d.ngroups * N;
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t) {
        if (16 * t < N) {
            if (nslice == 1) {
                store4(dq + at + 16 * t, aq[t][0], aq[t][1], aq[t][2], aq[t][3]);
                store4(dk + at + 16 * t, ak[t][0], ak[t][1], ak[t][2], ak[t][3]);
            } else {
                float* o = partial + slice * 2 * all + at + 16 * t;
                store4(o, aq[t][0], aq[t][1], aq[t][2], aq[t][3]);
                store4(o + all, ak[t][0], ak[t][1], ak[t][2], ak[t][3]);
            }
        }
    }
}

// dq and dk from the slices' partial sums, 4 elements a thread (n4 = elements / 4 of one of the two)
template <typename T>
__global__ __launch_bounds__(256) void delta_kq_sum_kernel(const float* __restrict__ partial, T* __restrict__ dq,
                                                           T* __restrict__ dk, int64_t n4, int nslice)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < 2 * n4; i += (int64_t)gridDim.x * 256) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < nslice; ++s) {
            const float4 b = reinterpret_cast<const float4*>(partial)[s * 2 * n4 + i];
            a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
        }
        T* o = i < n4 ? dq + 4 * i : dk + 4 * (i - n4);
        store4(o, a.x, a.y, a.z, a.w);
    }
}

// ---- host -----------------------------------------------------------------------------------------------------

// Head slices of the dq, dk step: enough workgroups to fill the GPU twice, at least 2 heads each.
int kq_slices(const DeltaDims& d)
{
    const int64_t wgs = d.seqs * ((d.seqlen + kChunk - 1) / kChunk) * d.ngroups, hpg = d.nheads / d.ngroups;
    if (wgs == 0) return 1;
    const int64_t want = (512 + wgs - 1) / wgs;
    return (int)(want < hpg / 2 ? want : hpg / 2 > 1 ? hpg / 2 : 1);
}

struct BwdSpace { size_t rec, x, w, ydy, sums, S, Slo, H, hs, part, total; };

BwdSpace bwd_space(const DeltaDims& d, size_t es)
{
    const size_t chunks = (d.seqlen + kChunk - 1) / kChunk, slots = delta_slots(d), heads = d.nheads;
    const size_t npt = d.headdim / 16, pn = d.headdim * ((d.dstate + 31) / 32 * 32), th = (size_t)d.seqs * heads * chunks * 64;
    const int ns = kq_slices(d);
    BwdSpace b;
    size_t at = 0;
    auto put = [&](size_t bytes) { const size_t here = at; at += (bytes + 255) / 256 * 256; return here; };
    b.rec = put(slots * heads * (es == 2 ? DeltaRec<bf16, true>::kBytes : DeltaRec<float, true>::kBytes));
    b.x = put(slots * heads * npt * 512 * 4);
    b.w = put(slots * heads * npt * 512 * es);
    b.ydy = put(npt * th * 4);
    b.sums = put(npt * th * 2 * 4);
    b.S = put((size_t)d.seqs * (chunks + 1) * heads * pn * es);
    b.Slo = put(es == 2 ? (size_t)d.seqs * (chunks + 1) * heads * pn * es : 0);
    b.H = put((size_t)d.seqs * chunks * heads * pn * es);
    b.hs = put(npt * (size_t)d.seqs * (chunks + 1) * heads * 4);
    b.part = put(ns > 1 ? (size_t)ns * 2 * d.tokens * d.ngroups * d.dstate * 4 : 0);
    b.total = at < 256 ? 256 : at;
    return b;
}

template <typename T, int NB, int NW>
hipError_t launch_rev(const T* v, const T* k, const T* q, const float* dfinal, const unsigned char* rec, T* dv,
                      float* dinit, const DeltaKeep<T>& keep, const DeltaBack<T>& back, const DeltaDims& d,
                      hipStream_t stream)
{
    const int nslice = (int)d.headdim / (16 * NW);
    const dim3 grid((unsigned)(d.seqs * d.nheads * nslice));
    constexpr unsigned kLds = RevCfg<T, NB, NW>::kBuf * RevCfg<T, NB, NW>::kStage;
    if constexpr (sizeof(T) == 2)
        hipLaunchKernelGGL((delta_rev_kernel<T, NB, NW>), grid, dim3(64 * NW), kLds, stream, v, k, q, dfinal, rec, dv,
                           dinit, keep, back, d, nslice);
    else
        hipLaunchKernelGGL((delta_rev_f32_kernel<T, NB, NW>), grid, dim3(64 * NW), kLds, stream, v, k, q, dfinal, rec, dv,
                           dinit, keep, back, d, nslice);
    return hipGetLastError();
}

template <typename T, int NB>
hipError_t launch_nb(const T* v, const float* g, const float* beta, const T* k, const T* q, const float* dfinal,
                     const unsigned char* rec, T* dv, T* dk, T* dq, float* dinit, float* partial,
                     const DeltaKeep<T>& keep, const DeltaBack<T>& back, const DeltaDims& d, hipStream_t stream)
{
    hipError_t e;
    if (d.headdim == 16) e = launch_rev<T, NB, 1>(v, k, q, dfinal, rec, dv, dinit, keep, back, d, stream);
    else if (d.headdim == 32 || sizeof(T) * NB == 32)
        e = launch_rev<T, NB, 2>(v, k, q, dfinal, rec, dv, dinit, keep, back, d, stream);
    else if constexpr (sizeof(T) * NB < 32)
        e = launch_rev<T, NB, 4>(v, k, q, dfinal, rec, dv, dinit, keep, back, d, stream);
    else e = hipErrorInvalidValue;
    if (e != hipSuccess || d.seqlen == 0) return e;
    const int ns = kq_slices(d);
    hipLaunchKernelGGL((delta_kq_kernel<T, NB>), dim3((unsigned)(d.seqs * keep.chunks * d.ngroups * ns)), dim3(256), 0,
                       stream, v, k, q, g, beta, keep, back, dq, dk, partial, d, ns);
    e = hipGetLastError();
    if (e != hipSuccess || ns == 1) return e;
    const int64_t n4 = d.tokens * d.ngroups * d.dstate / 4;
    hipLaunchKernelGGL((delta_kq_sum_kernel<T>), dim3((unsigned)(2 * n4 < (1 << 22) ? (2 * n4 + 255) / 256 : 1 << 14)),
                       dim3(256), 0, stream, partial,
                       dq, dk, n4, ns);
    return hipGetLastError();
}

}  // namespace

size_t delta_backward_workspace(const DeltaDims& d, int elem_bytes) { return bwd_space(d, (size_t)elem_bytes).total; }

template <typename T>
hipError_t launch_delta_backward(const T* v, const float* g, const float* beta, const T* k, const T* q,
                                 const float* init, const T* dy, const float* dfinal, T* dv, float* dg, float* dbeta,
                                 T* dk, T* dq, float* dinit, const DeltaDims& d, void* workspace, hipStream_t stream)
{
    if (d.seqs == 0) return hipSuccess;
    const BwdSpace b = bwd_space(d, sizeof(T));
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    auto f = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    auto t = [&](size_t at) { return reinterpret_cast<T*>(ws + at); };
    const int64_t chunks = (d.seqlen + kChunk - 1) / kChunk;
    const DeltaKeep<T> keep{dy, f(b.x), f(b.ydy), t(b.S), t(b.Slo), chunks};
    const DeltaBack<T> back{t(b.w), f(b.sums), t(b.H), f(b.hs)};
    hipError_t e = launch_delta_prep<T, true>(k, q, g, beta, ws + b.rec, d, stream);
    if (e == hipSuccess)
        e = launch_delta_chain<T, true>(v, k, q, init, ws + b.rec, nullptr, nullptr, keep, d, stream);
    if (e != hipSuccess) return e;
    if (d.dstate <= 32)
        e = launch_nb<T, 1>(v, g, beta, k, q, dfinal, ws + b.rec, dv, dk, dq, dinit, f(b.part), keep, back, d, stream);
    else if (d.dstate <= 64)
        e = launch_nb<T, 2>(v, g, beta, k, q, dfinal, ws + b.rec, dv, dk, dq, dinit, f(b.part), keep, back, d, stream);
    else if (d.dstate <= 128)
        e = launch_nb<T, 4>(v, g, beta, k, q, dfinal, ws + b.rec, dv, dk, dq, dinit, f(b.part), keep, back, d, stream);
    else
        e = launch_nb<T, 8>(v, g, beta, k, q, dfinal, ws + b.rec, dv, dk, dq, dinit, f(b.part), keep, back, d, stream);
    if (e != hipSuccess || d.seqlen == 0) return e;
    const int hblocks = (int)((d.nheads + 15) / 16);
    hipLaunchKernelGGL(delta_scalar_kernel, dim3((unsigned)(d.seqs * chunks * hblocks)), dim3(256), 0, stream, keep.ydy,
                       back.sums, back.hs, g, dg, dbeta, d, chunks, hblocks, init == nullptr ? 1 : 0);
    return hipGetLastError();
}

template hipError_t launch_delta_backward<float>(const float*, const float*, const float*, const float*, const float*,
                                                 const float*, const float*, const float*, float*, float*, float*,
                                                 float*, float*, float*, const DeltaDims&, void*, hipStream_t);
template hipError_t launch_delta_backward<bf16>(const bf16*, const float*, const float*, const bf16*, const bf16*,
                                                const float*, const bf16*, const float*, bf16*, float*, float*,
                                                bf16*, bf16*, float*, const DeltaDims&, void*, hipStream_t);

}  // namespace ssd
